// int8_tc.cu -- products of the 8-bit integer operators on the 5th-generation
// tensor cores.
//
// Mathematics.  D[r, c] = sum over k of a[r, k] b[c, k] with `a` 8-bit integers.
// The chip has no fast integer tensor instruction, but 16-bit floats hold
// 8-bit integers exactly and their products have at most 15 bits, so that
// kind::f16 with its 32-bit accumulator adds up to 1024 of them exactly
// (128 * 128 * 1024 = 2^24).  Integer sums are taken 1024 products at a time and
// added as integers.  A checkpoint's values q * u (q at most seven bits, u a
// power of two) are exact in 16 bits too.  The tensor core cuts off what is below
// the accumulator's last place, so a gradient's sums leave it every 512 tokens
// for 32-bit outputs, and for 16-bit ones before it shows (int8_most_tokens()); they
// are added up in registers.
//
// Structure.  Two CTAs on two SMs share a tile of 256 rows x kN columns
// (tcgen05.mma.cta_group::2): each supplies 128 rows of `a` and stages half of b's columns.
//  * warp 0 streams `a` (bytes, as they are in memory) and a checkpoint's units, warp
//    1 b, through two rings in shared memory (TMA, 128-byte swizzle);
//  * two groups of four warps take a's stages in turn, a row a lane: they turn
//    128 bytes into 16-bit floats in registers and write them to tensor
//    memory, from where the MMA takes its first operand.  Shared memory then moves 8
//    bits of `a` where 16 would pass twice, and no pass over `a` comes before;
//  * warp 2 of the pair's first CTA issues the MMAs;
//  * eight warps read a finished accumulator while the next one is filled.
// Where there are few tiles, pairs of one cluster take shares of k, and each adds up its part of the columns from the others'
// accumulators through shared memory: weight gradient 4096 x 1024 x 1024 bf16 14.2 us, with the shares written and added by
// join_kernel 16.6 (16384 tokens, 512 x 512, 20.4 and 16.8: more than four shares are left to that).
// Lanes are rows of D, which is stored as columns (out[c * ld + r]): a warp's 32
// values of a column are consecutive.
//
// What bounds it, measured.  16384 tokens, 4096 x 4096 (bfloat16, 256 columns): 313 us, 1756 TFLOP/s with the tensor pipe
// active 96 % of the time at the 1.78 GHz that power leaves; with 128 columns the converting warps bound it (390 us).
// 8192^3 of integers (128 columns, 8 runs a tile): 566 us, 1942 TFLOP/s, tensor pipe 87 %, L2 to SM 14.8 TB/s.  256 columns
// have one accumulator, so that a tile's (or a run's) sums are read before the next one's first product; that costs
// little after the 128 stages of a gradient's tile, 5 % after runs of 16 (16384 tokens, 4096 x 4096 bfloat16: runs of 4, 8, 16
// and 32 377, 348, 331 and 334 us, without any 313; runs of 4 in tiles of 128 columns 397), and much after the 8 of a run of
// integers, whose products have 128 columns and two accumulators.  With the first operand in tensor memory an MMA of 32 or 64 columns takes as long as one of 128
// (0.28 us a stage, 0.34 on every SM at once): small tiles only spread few columns over more SMs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "fp4_tc.cuh"
#include "int8_device.cuh"
#include "int8_internal.h"
#include "int8_plan.h"
#include "sgemm_device.cuh"
#include "sgemm_internal.h"

namespace gb300 {
namespace {

using namespace int8;
using fp4::elected;
using fp4::expect_bytes;
using fp4::load_box;
using fp4::operand_desc;
using fp4::uniform_warp;

constexpr uint32_t kStatusTimeout = 3;
constexpr int kStep = int(kInt8TcStep);
constexpr int kRows = 128;               // of a CTA
constexpr int kGroups = 2;               // of four warps that turn `a` to 16 bits

// kIntegers: 16-bit floats of integers, b K-major.  Others: a checkpoint's values in bfloat16 or 16-bit floats, b MN-major.
enum Kind { kIntegers, kBf16, kF16 };

template <Kind kKind_, int kN_, bool kRuns_>
struct Tile {
  static constexpr Kind kKind = kKind_;
  static constexpr int kN = kN_;
  static constexpr bool kRuns = kRuns_;  // sums leave the accumulator every `run` stages
  static constexpr bool kUnits = kKind != kIntegers;
  static constexpr bool kWideRuns = kRuns && kN == 256;  // the epilogue's sums take 128 registers a thread
  static constexpr int kCols = kN / 2;   // of b, a CTA
  static constexpr uint32_t kABytes = kRows * kStep, kUBytes = kUnits ? 1024 : 0, kBBytes = kCols * kStep * 2;
  static constexpr int kAccs = kN <= 128 ? 2 : 1;
  static constexpr int kSlotCols = kStep / 2;  // tensor memory columns of a stage of `a`
  static constexpr int kSlots0 = (512 - kAccs * kN) / kSlotCols;
  static constexpr int kSlots = kSlots0 < 6 ? kSlots0 : 6;
  // Shares of k of up to four pairs in a cluster meet where the stages were: each pair adds up its part of the columns.
  static constexpr int kMaxShares = kN <= 128 ? 4 : 1;  // (a warp's sums are in registers then)
  static constexpr int kStages0 = int((232448 - 1024 - 512) / (kABytes + kUBytes + kBBytes));
  static constexpr int kStages = kStages0 < 8 ? kStages0 : 8;
  static constexpr int kThreads = 128 * (3 + kGroups);
  static constexpr int kV = kN / 2;  // columns of an epilogue warp
  static constexpr int kBarriers = 4 * kStages + 2 * kSlots + 2 * kAccs + 1;
  static constexpr size_t kSmem = 1024 + kStages * size_t(kABytes + kUBytes + kBBytes) + kBarriers * 8 + 16;
  static_assert(kRows * kN * 4 <= kStages * (kABytes + kBBytes), "shares");
  static_assert(kSmem <= 232448 && kAccs * kN + kSlots * kSlotCols <= 512, "memory");
  // 32-bit accumulator; A from tensor memory, B K-major or MN-major (bit 16); M = 256.
  static constexpr uint32_t kDesc = (1u << 4) | (kKind == kBf16 ? (1u << 7) | (1u << 10) : 0u) | (kUnits ? 1u << 16 : 0u) |
                                    (uint32_t(kN >> 3) << 17) | (256u >> 4 << 24);
};

// The same place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t place_in(const void* p, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(dev::smem_addr(p)), "r"(rank));
  return d;
}
// What these arrivals hand over is in tensor memory and ordered by tcgen05.fence; with the release at cluster scope,
// which waits for all of the warp's earlier accesses, a stage took 3400 cycles instead of 1640.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrives on `bar` of the CTAs of `mask` once the tcgen05 operations issued so far completed.
__device__ __forceinline__ void commit(uint32_t e, uint64_t* bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
          dev::smem_addr(bar)),
      "h"(mask), "r"(e)
      : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void mma(uint32_t e, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(e)
      : "memory");
}

// MN-major rows of 128 bytes (64 columns) with the 128-byte swizzle: groups of eight k
// 1024 bytes apart, the next 64 columns kStep rows on.
__device__ __forceinline__ uint64_t columns_desc(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | uint64_t(kStep * 128 >> 4) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}

template <int kCount>
__device__ __forceinline__ void read_tmem(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int c = 0; c < kCount; c += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[c]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]), "=r"(r[c + 5]), "=r"(r[c + 6]),
          "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]), "=r"(r[c + 10]), "=r"(r[c + 11]), "=r"(r[c + 12]),
          "=r"(r[c + 13]), "=r"(r[c + 14]), "=r"(r[c + 15])
        : "r"(taddr + c));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void write_tmem32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]),
      "r"(taddr)
      : "memory");
}

// A place in a ring of kCount and the parity of its round.
template <int kCount>
struct At {
  uint32_t i = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == uint32_t(kCount)) i = 0, parity ^= 1u;
  }
};

// A unit of work: a tile and a range of its stages of k.
struct Work {
  int r0, c0, kb, ke, part;
};
__device__ __forceinline__ Work work_of(const Int8TcArgs& a, int unit, int kn) {
  const int tile = unit / a.splits, part = unit - tile * a.splits;
  // Tiles in bands of kBand rows of tiles, column by column, so that the pairs at work read few rows and columns.
  constexpr int kBand = 8;
  const int band = tile / (kBand * a.tiles_c), in_band = tile - band * kBand * a.tiles_c;
  const int height = min(kBand, a.tiles_r - band * kBand);
  const int tc = in_band / height, tr = band * kBand + in_band - tc * height;
  const int64_t all = a.steps;
  return {tr * 2 * kRows, tc * kn, int(all * part / a.splits), int(all * (part + 1) / a.splits), part};
}

template <typename T2>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  T2 v;
  v.x = from_f32<decltype(v.x)>(a);
  v.y = from_f32<decltype(v.y)>(b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// A unit's stages of b in their order: f(stage of k, term, whether an accumulator starts or ends with it).  A run's
// smaller terms come first: every addition cuts off what is below the accumulator's last place, and
// with the terms of a stage one after the other 4096 x 1024 x 1024 was 1.8e-6 off instead of 1.3e-7.
template <typename S, typename F>
__device__ __forceinline__ void for_stages(const Int8TcArgs& args, const Work& w, F f) {
  if (!S::kRuns || args.terms == 1) {
    int left = 0;  // stages until the accumulator changes
    for (int k = w.kb; k < w.ke; ++k) {
      const bool starts = left == 0;
      if (starts) left = S::kRuns ? min(args.run, w.ke - k) : w.ke - k;
      f(k, 0, starts, --left == 0);
    }
  } else {
    for (int k0 = w.kb; k0 < w.ke; k0 += args.run) {
      const int k1 = min(k0 + args.run, w.ke);
      for (int term = args.terms - 1; term >= 0; --term)
        for (int k = k0; k < k1; ++k) f(k, term, term == args.terms - 1 && k == k0, term == 0 && k + 1 == k1);
    }
  }
}

template <int kValue>
struct Int {
  __device__ constexpr operator int() const { return kValue; }
};
// f(0) .. f(kCount - 1), constants.
template <int kCount, int kFrom = 0, typename F>
__device__ __forceinline__ void for_parts(F f) {
  if constexpr (kFrom < kCount) {
    f(Int<kFrom>());
    for_parts<kCount, kFrom + 1>(f);
  }
}

// Stores kCount columns of a row of D (`out`: the first; `left`: those that exist), added to what is there if asked.
template <typename T, int kCount>
__device__ __forceinline__ void put_columns(T* out, int64_t ld, int left, bool add, const float (&v)[kCount]) {
  constexpr int kPart = kCount < 16 ? kCount : 16;
#pragma unroll
  for (int c0 = 0; c0 < kCount; c0 += kPart) {
    float old[kPart] = {};
    if (add) {
      const T* from = out;
#pragma unroll
      for (int c = 0; c < kPart; ++c, from += ld)
        if (c0 + c < left) old[c] = to_f32(*from);
    }
#pragma unroll
    for (int c = 0; c < kPart; ++c, out += ld)
      if (c0 + c < left) *out = from_f32<T>(add ? v[c0 + c] + old[c] : v[c0 + c]);
  }
}
template <int kCount>
__device__ __forceinline__ void put_columns(const Int8TcArgs& a, int64_t row, int col, const float (&v)[kCount]) {
  const int64_t at = int64_t(col) * a.ld + row;
  if (a.dtype == INT8_F32)
    put_columns(static_cast<float*>(a.out) + at, a.ld, a.cols - col, a.accumulate, v);
  else if (a.dtype == INT8_BF16)
    put_columns(static_cast<__nv_bfloat16*>(a.out) + at, a.ld, a.cols - col, a.accumulate, v);
  else
    put_columns(static_cast<__half*>(a.out) + at, a.ld, a.cols - col, a.accumulate, v);
}

// Stores kCount columns of a row, two 16-bit values in a register.  (The address is counted on from column to column: as
// c * ld from the first, the tiles of 4096 x 4096 x 1008 took 63 us instead of 25.)
template <int kCount>
__device__ __forceinline__ void put_pairs(uint16_t* out, int64_t ld, int left, const uint32_t (&two)[kCount / 2]) {
#pragma unroll
  for (int c = 0; c < kCount; c += 2) {
    if (c < left) out[0] = uint16_t(two[c / 2]);
    if (c + 1 < left) out[ld] = uint16_t(two[c / 2] >> 16);
    out += 2 * ld;
  }
}

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_u,
                   const __grid_constant__ CUtensorMap map_b, const Int8TcArgs args) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  unsigned char* s_a = smem;
  unsigned char* s_b = s_a + S::kStages * S::kABytes;
  unsigned char* s_u = s_b + S::kStages * S::kBBytes;
  uint64_t* a_full = reinterpret_cast<uint64_t*>(s_u + S::kStages * S::kUBytes);
  uint64_t* a_empty = a_full + S::kStages;
  uint64_t* b_full = a_empty + S::kStages;     // used in the first CTA
  uint64_t* b_empty = b_full + S::kStages;
  uint64_t* slot_full = b_empty + S::kStages;  // used in the first CTA
  uint64_t* slot_empty = slot_full + S::kSlots;
  uint64_t* acc_full = slot_empty + S::kSlots;
  uint64_t* acc_empty = acc_full + S::kAccs;   // used in the first CTA
  uint64_t* drain = acc_empty + S::kAccs;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1) + 1;

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t cluster_rank;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(cluster_rank));
  const uint32_t rank = cluster_rank & 1, leader = cluster_rank & ~1u;  // in the pair, and its first CTA
  const bool first = rank == 0;
  const uint16_t both = uint16_t(3u << leader);
  const int unit0 = blockIdx.x / 2, pairs = gridDim.x / 2;
  const uint64_t limit = args.wait_limit_ns;

  if (warp == 3) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     dev::smem_addr(const_cast<uint32_t*>(tmem_slot))), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      dev::mbar_init(&a_full[s], 1);
      dev::mbar_init(&a_empty[s], 4);
      dev::mbar_init(&b_full[s], 1);
      dev::mbar_init(&b_empty[s], 1);
    }
    for (int s = 0; s < S::kSlots; ++s) {
      dev::mbar_init(&slot_full[s], 8);
      dev::mbar_init(&slot_empty[s], 1);
    }
    for (int b = 0; b < S::kAccs; ++b) {
      dev::mbar_init(&acc_full[b], 1);
      dev::mbar_init(&acc_empty[b], 16);
    }
    dev::mbar_init(drain, 1);
    *s_abort = 0;
    dev::mbar_init_fence();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anything signals them
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  constexpr uint32_t tmem = fp4::kTmemBase, slots = tmem + S::kAccs * S::kN;
  // Whoever reads what the kernel before wrote waits for it, which is everybody unless that kernel only
  // prepared b and itself waited for the ones before: `a` can be read beside it then.
  const bool early = args.early && (warp == 0 || (warp >= 4 && warp < 4 + 4 * kGroups));
  if (!early) asm volatile("griddepcontrol.wait;" ::: "memory");

  auto fail = [&]() {
    if (!*s_abort) {
      *s_abort = 1;
      dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
    }
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dev::mbar_wait_abortable(bar, parity, limit, s_abort)) fail();
  };
  // After a failure, the copies in flight get a bounded time to land before shared memory is released.
  auto settle = [&]() {
    const uint64_t t0 = dev::global_timer_ns();
    while (dev::global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
  };
  auto going = [&]() { return __shfl_sync(0xffffffffu, *s_abort, 0) == 0; };

  // 640 threads have 96 registers each (61440); these four warps, and with 256 columns of runs the eight that turn `a`, give up
  // what the epilogue's sums need: 128 * 32 + 256 * 96 + 256 * 128, or 128 * 32 + 256 * 56 + 256 * 168.  (The eight do with 56; of
  // the epilogue's 11 do not fit beside its 128 sums, and more for it cannot be had.)
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    if (warp == 0) {
      // ---- `a` and its units, of this CTA's rows
      At<S::kStages> s;
      bool go = true;
      for (int unit = unit0; go && unit < args.units; unit += pairs) {
        const Work w = work_of(args, unit, S::kN);
        const int r0 = w.r0 + int(rank) * kRows;
        for (int k = w.kb; k < w.ke; ++k, s.next()) {
          wait(&a_empty[s.i], s.parity ^ 1u);  // (passes in the first round)
          if (!(go = going())) break;
          const uint32_t e = elected(), bar = dev::smem_addr(&a_full[s.i]);
          const int at = k * kStep;
          expect_bytes(e, &a_full[s.i], S::kABytes + S::kUBytes);
          load_box<1>(e, s_a + s.i * S::kABytes, &map_a, at, r0, bar);
          if constexpr (S::kUnits) {
            load_box<1>(e, s_u + s.i * S::kUBytes, &map_u, 2 * at, r0 / kBlock, bar);
            load_box<1>(e, s_u + s.i * S::kUBytes + 512, &map_u, 2 * at + 128, r0 / kBlock, bar);
          }
        }
      }
      if (!go) settle();
    } else if (warp == 1) {
      // ---- b, this CTA's half of the columns; completes on the first CTA's barrier
      At<S::kStages> s;
      bool go = true;
      for (int unit = unit0; go && unit < args.units; unit += pairs) {
        const Work w = work_of(args, unit, S::kN);
        const int c0 = w.c0 + int(rank) * S::kCols;
        for_stages<S>(args, w, [&](int k, int term, bool, bool) {
          if (go) {
            wait(&b_empty[s.i], s.parity ^ 1u);
            go = going();
          }
          if (go) {
            const uint32_t e = elected(), bar = place_in(&b_full[s.i], leader);
            if (first) expect_bytes(e, &b_full[s.i], 2 * S::kBBytes);
            unsigned char* to = s_b + s.i * S::kBBytes;
            if constexpr (S::kUnits) {
  #pragma unroll
              for (int j = 0; j < S::kCols / 64; ++j)
                load_box<2>(e, to + j * kStep * 128, &map_b, 2 * (c0 + 64 * j), k * kStep + term * args.depth, bar);
            } else {
  #pragma unroll
              for (int j = 0; j < 2; ++j) load_box<2>(e, to + j * S::kCols * 128, &map_b, 2 * kStep * k + 128 * j, c0, bar);
            }
            s.next();
          }
        });
      }
      if (!go) settle();
    } else if (warp == 2) {
      if (first) {
        // ---- MMAs.  The loop's own instructions have to be few: a stage's MMAs take 512 cycles with 128 columns.
        At<S::kSlots> t;
        At<S::kStages> s;
        At<S::kAccs> b;
        const uint64_t desc0 = S::kUnits ? columns_desc(dev::smem_addr(s_b)) : operand_desc(dev::smem_addr(s_b));
        for (int unit = unit0; unit < args.units; unit += pairs) {
          const Work w = work_of(args, unit, S::kN);
          At<S::kSlots> at = t;  // within the run
          for_stages<S>(args, w, [&](int k, int term, bool starts, bool ends) {
            const bool last = term == 0;  // of the stage's terms
            if (starts) wait(&acc_empty[b.i], b.parity ^ 1u);
            if (starts || (args.terms > 1 && (k - w.kb) % args.run == 0)) at = t;
            if (term == args.terms - 1) wait(&slot_full[at.i], at.parity);
            wait(&b_full[s.i], s.parity);
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint32_t d = tmem + b.i * S::kN, a = slots + at.i * S::kSlotCols, e = elected();
            const uint64_t db = desc0 + s.i * (S::kBBytes >> 4);
            uint32_t add = starts ? 0u : 1u;
  #pragma unroll
            for (int j = 0; j < kStep / 16; ++j) {
              mma(e, d, a + 8 * j, db + (S::kUnits ? j * (16 * 128 >> 4) : j / 4 * (S::kCols * 128 >> 4) + j % 4 * 2), S::kDesc, add);
              add = 1u;
            }
            commit(e, &b_empty[s.i], both);
            if (last) commit(e, &slot_empty[at.i], both);
            if (ends) {
              commit(e, &acc_full[b.i], both);
              b.next();
            }
            s.next();
            at.next();
            if (last) t = at;
          });
        }
        commit(elected(), drain, both);
        dev::mbar_wait(drain, 0u, limit);
      }
    }
  } else if (warp < 4 + 4 * kGroups) {
    // ---- `a` to 16 bits, in tensor memory
    if constexpr (S::kWideRuns) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    const int q = warp & 3, group = (warp - 4) >> 2, row = 32 * q + lane;
    const uint32_t to = slots + (uint32_t(32 * q) << 16);
    At<S::kStages> s;
    At<S::kSlots> t;
    int turn = 0;
    for (int unit = unit0; unit < args.units; unit += pairs) {
      const Work w = work_of(args, unit, S::kN);
      for (int k = w.kb; k < w.ke; ++k, s.next(), t.next()) {
        const bool mine = turn == group;
        if (++turn == kGroups) turn = 0;
        if (!mine) continue;
        wait(&a_full[s.i], s.parity);
        const uint4* from = reinterpret_cast<const uint4*>(s_a + s.i * S::kABytes + row * 128);
        const unsigned char* units = s_u + s.i * S::kUBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 in[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) in[j] = from[(4 * h + j) ^ (row & 7)];
          uint32_t out[32];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t word[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
            if constexpr (S::kUnits) {
              // 16 units, two 16-byte pieces of row q (its second 64 in the second box) of the swizzled boxes.
              uint32_t u[8];
#pragma unroll
              for (int p = 0; p < 2; ++p)
                *reinterpret_cast<uint4*>(u + 4 * p) = *reinterpret_cast<const uint4*>(
                    units + h * 512 + q * 128 + (((2 * j + p) ^ (q + 4 * h)) << 4));
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                if constexpr (S::kKind == kBf16) {
                  out[8 * j + 2 * x] = bmul2(to_bf16<0>(word[x]), u[2 * x]);
                  out[8 * j + 2 * x + 1] = bmul2(to_bf16<1>(word[x]), u[2 * x + 1]);
                } else {
                  const uint32_t v = word[x] ^ 0x80808080u;
                  out[8 * j + 2 * x] = hmul2(to_f16<0>(v), u[2 * x]);
                  out[8 * j + 2 * x + 1] = hmul2(to_f16<1>(v), u[2 * x + 1]);
                }
              }
            } else {
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t v = word[x] ^ 0x80808080u;
                out[8 * j + 2 * x] = to_f16<0>(v);
                out[8 * j + 2 * x + 1] = to_f16<1>(v);
              }
            }
          }
          if (h == 0) {
            wait(&slot_empty[t.i], t.parity ^ 1u);
            __syncwarp();
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          } else {
            __syncwarp();
            if (lane == 0) dev::mbar_arrive(&a_empty[s.i]);
          }
          write_tmem32(to + t.i * S::kSlotCols + 32 * h, out);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_at(place_in(&slot_full[t.i], leader));
      }
    }
  } else {
    if constexpr (S::kWideRuns)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    // ---- epilogue: 32 rows x kV columns a warp
    const int q = warp & 3, half = (warp - 4 - 4 * kGroups) >> 2;
    const uint32_t lanes = uint32_t(32 * q) << 16;
    At<S::kAccs> b;
    for (int unit = unit0; unit < args.units; unit += pairs) {
      const Work w = work_of(args, unit, S::kN);
      const int row = w.r0 + int(rank) * kRows + 32 * q + lane, col0 = w.c0 + half * S::kV;
      const bool mine = row < args.rows;
      constexpr int kPart = S::kWideRuns ? 16 : S::kV < 32 ? S::kV : 32;
      auto put_partials = [&](int c0, const uint32_t* bits) {
        uint32_t* out = args.partials + (int64_t(w.part) * args.cols + col0 + c0) * args.rows + row;
#pragma unroll
        for (int c = 0; c < kPart; ++c, out += args.rows)
          if (mine && col0 + c0 + c < args.cols) *out = bits[c];
      };
      auto acc_wait = [&]() {
        wait(&acc_full[b.i], b.parity);
        __syncwarp();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        return tmem + b.i * S::kN + half * S::kV + lanes;
      };
      auto acc_free = [&]() {
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) arrive_at(place_in(&acc_empty[b.i], leader));
        b.next();
      };
      if constexpr (S::kRuns || S::kMaxShares > 1) {
        if (S::kRuns || args.join) {
          // Scales of this warp's columns, 32 a register; a row's.
          float scale_c[(S::kV + 31) / 32], scale_r = 0.f;
          if (S::kKind == kIntegers && (args.splits == 1 || args.join)) {
#pragma unroll
            for (int c = 0; c < S::kV; c += 32) scale_c[c / 32] = col0 + c + lane < args.cols ? args.scale_c[col0 + c + lane] : 0.f;
            if (mine) scale_r = args.scale_r[row];
          }
          uint32_t sum[S::kV];
          if constexpr (S::kRuns) {
#pragma unroll
            for (int c = 0; c < S::kV; ++c) sum[c] = 0;
            for (int k = w.kb; k < w.ke; k += args.run) {
              const uint32_t at = acc_wait();
#pragma unroll
              for (int c = 0; c < S::kV; c += kPart) {
                float v[kPart];
                read_tmem<kPart>(at + c, v);
#pragma unroll
                for (int x = 0; x < kPart; ++x)
                  sum[c + x] = S::kKind == kIntegers ? sum[c + x] + uint32_t(__float2int_rn(v[x]))
                                                     : __float_as_uint(__uint_as_float(sum[c + x]) + v[x]);
              }
              acc_free();
            }
          } else {
            read_tmem<S::kV>(acc_wait(), reinterpret_cast<float*>(sum));
            acc_free();
          }
          const bool ok = going();
          // Stores n of the columns from c on.
          auto store = [&](auto c, auto n) {
            float v[n];
#pragma unroll
            for (int x = 0; x < n; ++x)
              v[x] = S::kKind == kIntegers ? scaled(int(sum[c + x]), scale_r, __shfl_sync(0xffffffffu, scale_c[(c + x) / 32], (c + x) % 32))
                                           : __uint_as_float(sum[c + x]);
            if (args.dtype != INT8_F32 && !args.accumulate) {
              uint32_t two[n / 2];
#pragma unroll
              for (int x = 0; x < n; x += 2) two[x / 2] = args.dtype == INT8_BF16 ? pack2<__nv_bfloat162>(v[x], v[x + 1]) : pack2<__half2>(v[x], v[x + 1]);
              if (mine) put_pairs<n>(static_cast<uint16_t*>(args.out) + int64_t(col0 + c) * args.ld + row, args.ld, args.cols - col0 - c, two);
            } else if (mine) {
              put_columns(args, row, col0 + c, v);
            }
          };
          // The only unit of this pair, one of kShares in the cluster: of the columns each pair has a part to add up and store.
          auto meet = [&](auto shares) {
            constexpr int kShares = shares, kOwn = S::kV / kShares;
            const int at = half * kOwn * kRows + 32 * q + lane;
            cluster_sync();  // everybody's products are done: nothing uses the stages any more
            if (ok) {
              for_parts<kShares>([&](auto o) {
                if (o == w.part) return;
                const uint32_t to = place_in(smem + (w.part - (w.part > o)) * (2 * kOwn * kRows * 4), 2 * o + rank) + 4 * at;
#pragma unroll
                for (int c = 0; c < kOwn; ++c)
                  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 4 * kRows * c), "r"(sum[o * kOwn + c]) : "memory");
              });
            }
            __syncwarp();
            cluster_sync();
            if (!ok) return;
            for_parts<kShares>([&](auto o) {
              if (o != w.part) return;
#pragma unroll
              for (int p = 0; p + 1 < kShares; ++p) {
                const uint32_t* from = reinterpret_cast<const uint32_t*>(smem) + p * (2 * kOwn * kRows) + at;
#pragma unroll
                for (int c = 0; c < kOwn; ++c) {
                  uint32_t& to = sum[o * kOwn + c];
                  to = S::kKind == kIntegers ? to + from[kRows * c] : __float_as_uint(__uint_as_float(to) + __uint_as_float(from[kRows * c]));
                }
              }
              store(Int<o * kOwn>(), Int<kOwn>());
            });
          };
          if (S::kMaxShares > 1 && args.join) {
            if constexpr (S::kMaxShares > 1) {
              if (args.splits == 2)
                meet(Int<2>());
              else
                meet(Int<4>());
            }
          } else if (ok) {
            for_parts<S::kV / kPart>([&](auto i) {
              if (args.splits > 1)
                put_partials(i * kPart, sum + i * kPart);
              else
                store(Int<i * kPart>(), Int<kPart>());
            });
          }
          continue;
        }
      }
      if constexpr (!S::kRuns) {
        const uint32_t at = acc_wait();
        const bool ok = going();
        if (args.splits > 1) {
#pragma unroll
          for (int c = 0; c < S::kV; c += kPart) {
            uint32_t v[kPart];
            read_tmem<kPart>(at + c, reinterpret_cast<float*>(v));
            if (ok) put_partials(c, v);
          }
          acc_free();
        } else if (args.accumulate) {
#pragma unroll
          for (int c = 0; c < S::kV; c += kPart) {
            float v[kPart];
            read_tmem<kPart>(at + c, v);
            if (ok && mine) put_columns(args, row, col0 + c, v);
          }
          acc_free();
        } else {
          // Rounded to the 16-bit type as they are read, so that the accumulator is free before the stores.
          uint32_t two[S::kV / 2];
#pragma unroll
          for (int c = 0; c < S::kV; c += kPart) {
            float v[kPart];
            read_tmem<kPart>(at + c, v);
#pragma unroll
            for (int x = 0; x < kPart; x += 2) two[(c + x) / 2] = args.dtype == INT8_BF16 ? pack2<__nv_bfloat162>(v[x], v[x + 1]) : pack2<__half2>(v[x], v[x + 1]);
          }
          acc_free();
          if (ok && mine) put_pairs<S::kV>(static_cast<uint16_t*>(args.out) + int64_t(col0) * args.ld + row, args.ld, args.cols - col0, two);
        }
      }
    }
  }
  __syncwarp();
  if (S::kMaxShares > 1 && args.join && warp < 4 + 4 * kGroups) cluster_sync(), cluster_sync();  // (the epilogue's warps were there)
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // nothing of any CTA is still signalled or read by another
  if (warp == 3) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Adds the shares of a product split over k, in their order, and stores it: kJoin columns of a row a thread.
constexpr int kJoin = 2;
template <bool kWhole>
__global__ void __launch_bounds__(256) join_kernel(const Int8TcArgs args) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int r = blockIdx.x * 256 + threadIdx.x, c0 = blockIdx.y * kJoin;
  if (r >= args.rows) return;
  const int64_t all = int64_t(args.rows) * args.cols;
  const uint32_t* from = args.partials + int64_t(c0) * args.rows + r;
  uint32_t sum[kJoin] = {};
#pragma unroll 4
  for (int p = 0; p < args.splits; ++p, from += all) {
    uint32_t x[kJoin];
#pragma unroll
    for (int c = 0; c < kJoin; ++c) x[c] = c0 + c < args.cols ? from[int64_t(c) * args.rows] : 0u;
#pragma unroll
    for (int c = 0; c < kJoin; ++c)
      sum[c] = kWhole ? sum[c] + x[c] : __float_as_uint(__uint_as_float(sum[c]) + __uint_as_float(x[c]));
  }
  float v[kJoin];
#pragma unroll
  for (int c = 0; c < kJoin; ++c)
    v[c] = kWhole ? (c0 + c < args.cols ? scaled(int(sum[c]), args.scale_r[r], args.scale_c[c0 + c]) : 0.f) : __uint_as_float(sum[c]);
  put_columns(args, r, c0, v);
}

typedef void (*Kernel)(CUtensorMap, CUtensorMap, CUtensorMap, Int8TcArgs);
struct Instance {
  Kernel kernel;
  size_t smem;
  int threads;
};
template <int kShape, Kind kKind, int kN, bool kRuns>
Instance instance_of() {
  using S = Tile<kKind, kN, kRuns>;
  constexpr Int8TcForm kForm = int8_tc_form(kShape);
  static_assert(kForm.cols == kN && kForm.shares == S::kMaxShares && (kForm.run > 0) == kRuns, "what plans are made with");
  static_assert(!kForm.terms || (kRuns && S::kSlots >= kForm.run), "a run's stages of `a` stay until its last term");
  return {Kernel(product_kernel<S>), S::kSmem, S::kThreads};
}

Instance instance(int shape) {
  switch (shape) {
    case kInt8Whole32: return instance_of<kInt8Whole32, kIntegers, 32, true>();
    case kInt8Whole64: return instance_of<kInt8Whole64, kIntegers, 64, true>();
    case kInt8Whole128: return instance_of<kInt8Whole128, kIntegers, 128, true>();
    case kInt8Bf16N128: return instance_of<kInt8Bf16N128, kBf16, 128, false>();
    case kInt8Bf16N256: return instance_of<kInt8Bf16N256, kBf16, 256, false>();
    case kInt8Bf16Runs: return instance_of<kInt8Bf16Runs, kBf16, 128, true>();
    case kInt8Bf16Runs256: return instance_of<kInt8Bf16Runs256, kBf16, 256, true>();
    case kInt8F16N128: return instance_of<kInt8F16N128, kF16, 128, false>();
    case kInt8F16N256: return instance_of<kInt8F16N256, kF16, 256, false>();
    case kInt8F16Runs256: return instance_of<kInt8F16Runs256, kF16, 256, true>();
    default: return instance_of<kInt8F16Runs, kF16, 128, true>();
  }
}

}  // namespace

bool int8_tc_prepare(Int8TcClusters* n) {
  Int8LeastClusters least;
  for (int shape = 0; shape < kInt8TcShapes; ++shape) {
    const Instance in = instance(shape);
    if (cudaFuncSetAttribute(reinterpret_cast<const void*>(in.kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(in.smem)) != cudaSuccess)
      return false;
    for (int pairs = 1; pairs <= int8_tc_form(shape).shares; pairs *= 2) {
      cudaLaunchAttribute attr = {};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = unsigned(2 * pairs);
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(unsigned(2 * pairs), 1, 1);
      cfg.blockDim = dim3(in.threads, 1, 1);
      cfg.dynamicSmemBytes = in.smem;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int most = 0;
      if (cudaOccupancyMaxActiveClusters(&most, reinterpret_cast<const void*>(in.kernel), &cfg) != cudaSuccess) return false;
      least.take(pairs, most);
    }
  }
  *n = least.clusters();
  return n->pairs > 0;
}

cudaError_t launch_int8_tc(Int8TcShape shape, const CUtensorMap (&maps)[3], const Int8TcArgs& args, int pairs,
                           cudaStream_t stream) {
  const Instance in = instance(shape);
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(args.join ? 2 * args.splits : 2);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(2 * (args.join ? args.units : std::min(pairs, args.units))), 1, 1);
  cfg.blockDim = dim3(unsigned(in.threads), 1, 1);
  cfg.dynamicSmemBytes = in.smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, in.kernel, maps[0], maps[1], maps[2], args);
  if (e != cudaSuccess || args.splits == 1 || args.join) return e;
  cfg.numAttrs = 1;  // no clusters
  // (Fewer tiles than pairs of CTAs were split: the columns are some ten thousand at most.)
  cfg.gridDim = dim3(unsigned((args.rows + 255) / 256), unsigned((args.cols + kJoin - 1) / kJoin), 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, args.scale_r ? join_kernel<true> : join_kernel<false>, args);
}

}  // namespace gb300
