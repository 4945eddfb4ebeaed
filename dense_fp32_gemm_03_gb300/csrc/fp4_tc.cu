// fp4_tc.cu -- products of 4-bit matrices on the 5th-generation tensor cores.
//
// Mathematics.  D[r, c] = sum over blocks of uR uC sum over the block of
// qR qC, which tcgen05.mma computes for packed 4-bit operands with one scale
// byte per block of each operand (kind::mxf4 for blocks of 32 with power-of-two
// scales, kind::mxf4nvf4 for blocks of 16 with 8-bit float scales), 64 columns
// of K an instruction (the chip has instructions of 96 at 1.5 times the rate, which are not
// used here), in 32-bit accumulators.  The factors of the two matrices
// multiply the finished sum.  One operand ("rows") supplies 128 rows a CTA, the
// other ("columns") kN.
//
// Structure, for one CTA or (kCtas = 2) a pair of CTAs on two SMs that share
// one 256-row tile and each stage half of its columns:
//  * warp 0 streams 256-column slices of K of both operands (TMA, 128-byte
//    swizzle) and of their scales (TMA, 512-byte atoms) through a ring;
//  * warp 1 (of the pair's first CTA) copies a slice's scales to tensor memory
//    (tcgen05.cp) and issues its four tcgen05.mma.  Scales have a place in
//    tensor memory for each stage of the ring, so a stage's barrier covers
//    them too;
//  * the epilogue warps read an accumulator into registers, give it back, and
//    store it or join it with the other shares of a tile split over K
//    (published in the workspace, added in CTA order by the last to arrive).
//
// What bounds it, measured.  A pair's 256 x 256 tile takes 34.8 KB a 256-column slice
// into each SM for 4 x 256 x 256 x 64 products, so that 8192^3 (nvfp4 to bf16, 166 us,
// 6.6 PFLOP/s) runs the tensor pipe 77 % of the time; L2 feeds an SM about 64 bytes a
// clock meanwhile, which is what a 128 x 128 tile of a single CTA takes for half the
// products (213 us).  The rest is a tile's accumulator, read before the next tile's
// first product since two do not fit beside the scales (7 %), and the stores.  A pair's
// 256 x 128 tile has two accumulators and fills a last wave better (4096^3 29.2 us, 32.0
// with 256 columns).  A deeper ring is worth more than a second store buffer: one stage
// less costs 256 x 128 tiles 5 % at 8192^3.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp4_tc.cuh"
#include "sgemm_device.cuh"
#include "sgemm_internal.h"
#include "sgemm_sched.cuh"

namespace gb300 {
namespace {

using namespace fp4;

constexpr uint32_t kStatusTimeout = 3;
constexpr uint32_t kSliceBytes = 128;  // of one row of codes: 256 columns of K, a stage

// One instance's shape and memory.
template <int kFormat, int kCtas_, int kN_>
struct Tile {
  static constexpr int kCtas = kCtas_, kN = kN_;
  static constexpr int kAtoms = Format<kFormat>::kAtomsPerStage;
  static constexpr int kRows = 128;             // of a CTA
  static constexpr int kBM = kRows * kCtas;     // of a tile
  static constexpr int kCols = kN / kCtas;      // columns that a CTA stages
  static constexpr int kColTiles = (kN + 127) / 128;  // 128-row scale tiles of the column operand
  static constexpr uint32_t kRBytes = kRows * kSliceBytes, kCBytes = kCols * kSliceBytes;
  static constexpr uint32_t kRScale = kAtoms * 512, kCScale = kAtoms * 512 * kColTiles;
  static constexpr uint32_t kStageBytes = kRBytes + kCBytes + kRScale + kCScale;
  static constexpr int kEpiWarps = kN > 128 ? 8 : 4;
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  static constexpr int kWarpCols = kN / (kEpiWarps / 4);  // accumulator columns of an epilogue warp
  static constexpr uint32_t kStaging = kN >= 128 ? kEpiWarps * 4096 : 0;  // one block an epilogue warp
  // Tensor memory: accumulators, then the scales of every stage.
  static constexpr int kScaleCols = kAtoms * 4 * (1 + kColTiles);
  static constexpr int kFit = int((232448 - 1024 - 512 - kStaging) / kStageBytes);
  static constexpr int kFitTmem = (512 - kN) / kScaleCols;
  static constexpr int kStages0 = kFit < kFitTmem ? kFit : kFitTmem;
  static constexpr int kStages = kStages0 < 8 ? kStages0 : 8;
  static constexpr int kAccs = 512 - kStages * kScaleCols >= 2 * kN ? 2 : 1;
  static constexpr int kScaleBase = kAccs * kN;  // first scale column
  static constexpr size_t kSmem = 1024 + kStages * size_t(kStageBytes) + kStaging + (2 * kStages + 5) * 8 + 16;
  static_assert(kSmem <= 232448 && kStages >= 3, "shared memory");
  static_assert(kScaleBase + kStages * kScaleCols <= 512, "tensor memory");
};

template <int kCtas>
__device__ __forceinline__ uint32_t barrier_of_first(uint64_t* bar) {
  if constexpr (kCtas == 1) return dev::smem_addr(bar);
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(dev::smem_addr(bar)), "r"(0));
  return d;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int kCount>
__device__ __forceinline__ void read_tmem(uint32_t taddr, float (&v)[kCount]) {
  static_assert(kCount % 16 == 0, "");
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

// The units of one CTA (pair): its share of the tiles split over K first, whose
// joining then runs beside the whole tiles' products.
struct UnitIter {
  WorkIter w;
  int dp_first;
  bool shares;

  __device__ __forceinline__ void init(const Sched& sc, int cta) {
    w.init(sc, cta);
    dp_first = w.dp_next;
    w.dp_next = sc.dp_tiles;
    shares = true;
  }
  __device__ __forceinline__ bool next(const Sched& sc, int ctas, Unit& u) {
    if (shares) {
      if (w.next(sc, ctas, u)) return true;
      shares = false;
      w.dp_next = dp_first;
    }
    return w.next(sc, ctas, u);
  }
};

// kSwap: the row operand is B, so D is C transposed and a lane's value goes to
// column `row` of C; otherwise lane = row of C, and blocks of 32 rows x 128
// bytes leave through shared memory.
template <typename T, int kFormat, int kCtas, int kN, bool kSwap>
__device__ __forceinline__ void tc_body(const CUtensorMap& map_r, const CUtensorMap& map_c,
                                        const CUtensorMap& map_rs, const CUtensorMap& map_cs,
                                        const CUtensorMap& map_out, const Fp4TcArgs& args, const Sched& sc) {
  using S = Tile<kFormat, kCtas, kN>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = dev::smem_addr(smem_raw);
  unsigned char* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  unsigned char* s_r = smem;
  unsigned char* s_c = s_r + S::kStages * S::kRBytes;
  unsigned char* s_out = s_c + S::kStages * S::kCBytes;  // 1024-byte aligned where it is used
  unsigned char* s_rs = s_out + S::kStaging;
  unsigned char* s_cs = s_rs + S::kStages * S::kRScale;
  uint64_t* full = reinterpret_cast<uint64_t*>(s_cs + S::kStages * S::kCScale);
  uint64_t* empty = full + S::kStages;
  uint64_t* acc_full = empty + S::kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;       // [2], used in the first CTA
  uint64_t* drain = acc_empty + 2;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(drain + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(drain + 1) + 1;
  int* s_last = reinterpret_cast<int*>(drain + 1) + 2;

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  uint32_t rank = 0;
  if constexpr (kCtas == 2) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const bool first = rank == 0;
  const int unit_id = blockIdx.x / kCtas, units = gridDim.x / kCtas;
  const uint64_t limit = args.wait_limit_ns;

  if (warp == 1) {
    if constexpr (kCtas == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       dev::smem_addr(const_cast<uint32_t*>(tmem_slot))), "r"(512u) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       dev::smem_addr(const_cast<uint32_t*>(tmem_slot))), "r"(512u) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      dev::mbar_init(&full[s], 1);
      dev::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      dev::mbar_init(&acc_full[b], 1);
      dev::mbar_init(&acc_empty[b], kCtas * S::kEpiWarps);
    }
    dev::mbar_init(drain, 1);
    *s_abort = 0;
    dev::mbar_init_fence();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();  // the peer's barriers exist before anything signals them
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  constexpr uint32_t tmem = kTmemBase;
  // The kernel before on the stream may still run up to here (300 x 520 x 200 in a graph 5.0 -> 4.6 us).
  asm volatile("griddepcontrol.wait;" ::: "memory");

  auto fail = [&]() {
    if (!*s_abort) {
      *s_abort = 1;
      dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
    }
  };

  if (warp == 0) {
    // ---- producer (both CTAs): completes on the first CTA's barrier
    if (dev::elect_one()) {
      dev::tma_prefetch_desc(&map_r);
      dev::tma_prefetch_desc(&map_c);
      dev::tma_prefetch_desc(&map_rs);
      dev::tma_prefetch_desc(&map_cs);
    }
    UnitIter w;
    w.init(sc, unit_id);
    Unit u;
    uint32_t i = 0;
    const int atoms = sc.iters_per_tile * S::kAtoms;  // of one 128-row scale tile
    bool go = true;
    while (go && w.next(sc, units, u)) {
      int tm, tn;
      tile_coords(sc, u.tile, tm, tn);
      const int r0 = tm * S::kBM + int(rank) * S::kRows, c0 = tn * kN + int(rank) * S::kCols;
      const int rs0 = (r0 >> 7) * atoms, cs0 = (tn * kN >> 7) * atoms;
      for (int k = u.kb; k < u.ke; ++k, ++i) {
        const uint32_t s = i % S::kStages, n = i / S::kStages;
        if (n > 0 && !dev::mbar_wait_abortable(&empty[s], (n - 1) & 1u, limit, s_abort)) fail();
        go = __shfl_sync(0xffffffffu, *s_abort, 0) == 0;
        if (!go) break;
        const uint32_t bar = barrier_of_first<kCtas>(&full[s]), e = elected();
        if (first) expect_bytes(e, &full[s], kCtas * S::kStageBytes);
        load_box<kCtas>(e, s_r + s * S::kRBytes, &map_r, k * int(kSliceBytes), r0, bar);
        load_box<kCtas>(e, s_c + s * S::kCBytes, &map_c, k * int(kSliceBytes), c0, bar);
        load_box<kCtas>(e, s_rs + s * S::kRScale, &map_rs, 0, rs0 + k * S::kAtoms, bar);
#pragma unroll
        for (int t = 0; t < S::kColTiles; ++t)
          load_box<kCtas>(e, s_cs + s * S::kCScale + t * S::kAtoms * 512, &map_cs, 0, cs0 + t * atoms + k * S::kAtoms, bar);
      }
    }
    // After a failure, the copies in flight get a bounded time to land (they
    // complete on the first CTA's barrier) before shared memory is released.
    if (!go) {
      const uint64_t t0 = dev::global_timer_ns();
      while (dev::global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
    }
  } else if (warp == 1) {
    if (first) {
      // ---- scales and MMAs (first CTA only)
      UnitIter w;
      w.init(sc, unit_id);
      Unit u;
      uint32_t it = 0, ui = 0;
      while (w.next(sc, units, u)) {
        const uint32_t b = ui % S::kAccs, nb = ui / S::kAccs;
        if (nb > 0 && !dev::mbar_wait_abortable(&acc_empty[b], (nb - 1) & 1u, limit, s_abort)) fail();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d = tmem + b * kN;
        int tm, tn;
        tile_coords(sc, u.tile, tm, tn);
        const uint32_t shift = uint32_t(tn * kN & 127) >> 5;  // the tile's first scale column in its 128-row tile
        for (int k = u.kb; k < u.ke; ++k, ++it) {
          const uint32_t s = it % S::kStages;
          if (!dev::mbar_wait_abortable(&full[s], (it / S::kStages) & 1u, limit, s_abort)) fail();
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t e = elected();
          const uint32_t sr = tmem + S::kScaleBase + s * S::kScaleCols, scl = sr + 4 * S::kAtoms;
          const uint64_t drs = scale_desc(dev::smem_addr(s_rs + s * S::kRScale));
          const uint64_t dcs = scale_desc(dev::smem_addr(s_cs + s * S::kCScale));
#pragma unroll
          for (int a = 0; a < S::kAtoms; ++a) {
            copy_scales<kCtas>(e, sr + 4 * a, drs + 32 * a);
#pragma unroll
            for (int t = 0; t < S::kColTiles; ++t)
              copy_scales<kCtas>(e, scl + 4 * (a * S::kColTiles + t), dcs + 32 * (t * S::kAtoms + a));
          }
          const uint64_t dr = operand_desc(dev::smem_addr(s_r + s * S::kRBytes));
          const uint64_t dc = operand_desc(dev::smem_addr(s_c + s * S::kCBytes));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            constexpr int kPer = 4 / S::kAtoms;  // MMAs that share an atom
            const int a = j / kPer;
            mma<kFormat, kCtas>(e, d, dr + 2 * j, dc + 2 * j,
                                instr_desc<kFormat>(128 * kCtas, kN, kPer == 2 ? (j & 1) * 2 : 0), sr + 4 * a,
                                scl + 4 * a * S::kColTiles + shift, (k != u.kb || j != 0) ? 1u : 0u);
          }
          commit<kCtas>(e, &empty[s]);
        }
        commit<kCtas>(elected(), &acc_full[b]);
        ++ui;
      }
      commit<kCtas>(elected(), drain);
      dev::mbar_wait(drain, 0u, limit);
    }
  } else {
    // ---- epilogue (both CTAs)
    constexpr int kV = S::kWarpCols;
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row_local = 32 * q + lane, col_local = half * kV;
    const int etid = threadIdx.x - 64;
    constexpr int64_t kSlot = int64_t(S::kRows) * kN / 4;  // one CTA's share of a tile, in float4
    float2 alpha = make_float2(1.f, 1.f);
    if (kFormat == FP4_NVFP4)
      alpha = join_factors(args.factor_r ? __ldg(args.factor_r) : 1.f, args.factor_c ? __ldg(args.factor_c) : 1.f);
    UnitIter w;
    w.init(sc, unit_id);
    Unit u;
    uint32_t ui = 0;
    while (w.next(sc, units, u)) {
      const uint32_t b = ui % S::kAccs, nb = ui / S::kAccs;
      if (!dev::mbar_wait_abortable(&acc_full[b], nb & 1u, limit, s_abort)) fail();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      int tm, tn;
      tile_coords(sc, u.tile, tm, tn);
      const bool ok = __shfl_sync(0xffffffffu, !*s_abort ? 1 : 0, 0) != 0;
      float v[kV];
      read_tmem<kV>(tmem + b * kN + col_local + (uint32_t(32 * q) << 16), v);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         barrier_of_first<kCtas>(&acc_empty[b])) : "memory");
      bool store = true;
      if (u.t_sk >= 0 && !(u.kb == 0 && u.ke == sc.iters_per_tile)) {
        // A share of a split tile.  The first share stays in registers if all
        // others have already arrived.
        const int64_t at = int64_t(u.t_sk) * sc.iters_per_tile;
        const int c_first = sk_owner(sc, at), c_last = sk_owner(sc, at + sc.iters_per_tile - 1);
        const int others = c_last - c_first;
        int32_t* counter = args.counters + kCtas * u.t_sk + int(rank);
        const bool mine_first = unit_id == c_first;
        bool last = false;
        if (mine_first) {
          if (etid == 0) *s_last = dev::ld_acquire_gpu(counter) == others ? 1 : 0;
          dev::named_barrier(1, 32 * S::kEpiWarps);
          last = *s_last != 0;
          dev::named_barrier(1, 32 * S::kEpiWarps);
        }
        float4* slot = reinterpret_cast<float4*>(args.partials) + int(rank) * kSlot + col_local / 4 * S::kRows + row_local;
        const bool kept = last;
        if (!last) {
          float4* mine = slot + int64_t(u.t_sk + unit_id) * kCtas * kSlot;
#pragma unroll
          for (int c = 0; c < kV / 4; ++c)
            __stcg(mine + c * S::kRows, make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]));
          dev::named_barrier(1, 32 * S::kEpiWarps);
          if (etid == 0) {
            __threadfence();
            *s_last = atomicAdd(counter, 1) == others ? 1 : 0;
            __threadfence();
          }
          dev::named_barrier(1, 32 * S::kEpiWarps);
          last = *s_last != 0;
          dev::named_barrier(1, 32 * S::kEpiWarps);
        }
        store = last;
        if (last) {
          // Sum in CTA order, whoever adds: the first share from registers or from its slot.
          if (!kept) {
            const float4* src = slot + int64_t(u.t_sk + c_first) * kCtas * kSlot;
#pragma unroll
            for (int c = 0; c < kV / 4; ++c) {
              const float4 x = __ldcg(src + c * S::kRows);
              v[4 * c] = x.x, v[4 * c + 1] = x.y, v[4 * c + 2] = x.z, v[4 * c + 3] = x.w;
            }
          }
#pragma unroll 1
          for (int o = c_first + 1; o <= c_last; ++o) {
            const float4* src = slot + int64_t(u.t_sk + o) * kCtas * kSlot;
#pragma unroll
            for (int c = 0; c < kV / 4; ++c) {
              const float4 x = __ldcg(src + c * S::kRows);
              v[4 * c] += x.x, v[4 * c + 1] += x.y, v[4 * c + 2] += x.z, v[4 * c + 3] += x.w;
            }
          }
          if (etid == 0) *counter = 0;
        }
      }
      if (store && ok) {
#pragma unroll
        for (int c = 0; c < kV; ++c) v[c] = v[c] * alpha.x * alpha.y;
        const int row = tm * S::kBM + int(rank) * S::kRows + row_local, col0 = tn * kN + col_local;
        T* out = static_cast<T*>(args.out);
        if constexpr (kSwap) {
          if (row < args.rows) {
#pragma unroll
            for (int c = 0; c < kV; ++c)
              if (col0 + c < args.cols) out[int64_t(col0 + c) * args.ld + row] = from_f32<T>(v[c]);
          }
        } else {
          constexpr int kPer = 128 / sizeof(T);  // columns of a block
          unsigned char* buf = s_out + (warp - 2) * 4096;
          const int row0 = row - lane;
#pragma unroll
          for (int c = 0; c < kV; c += kPer) {
            if (col0 + c >= args.cols || row0 >= args.rows) break;
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
            // 16-byte piece j of row r at j ^ (r mod 8): what TMA reads with the 128-byte swizzle.
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint4 piece;
              T* t = reinterpret_cast<T*>(&piece);
#pragma unroll
              for (int e = 0; e < kPer / 8; ++e) t[e] = from_f32<T>(v[c + j * (kPer / 8) + e]);
              reinterpret_cast<uint4*>(buf + lane * 128)[j ^ (lane & 7)] = piece;
            }
            // A TMA store clips a box at the right edge to 16-byte pieces only.
            if (args.tma_out && (args.tma_edge || col0 + c + kPer <= args.cols)) {
              dev::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                                 reinterpret_cast<uint64_t>(&map_out)),
                             "r"((col0 + c) * int(sizeof(T))), "r"(row0), "r"(dev::smem_addr(buf))
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
              }
            } else {
              __syncwarp();
              // Eight rows' reads before their stores: one row at a time waits out each read.
#pragma unroll 1
              for (int r0 = 0; r0 < 32; r0 += 8)
#pragma unroll
                for (int e = lane; e < kPer; e += 32) {
                  T t[8];
#pragma unroll
                  for (int r = 0; r < 8; ++r)
                    t[r] = reinterpret_cast<const T*>(buf + (r0 + r) * 128)[((e / (kPer / 8)) ^ r) * (kPer / 8) + e % (kPer / 8)];
                  T* at = out + int64_t(row0 + r0) * args.ld + col0 + c + e;
#pragma unroll
                  for (int r = 0; r < 8; ++r)
                    if (col0 + c + e < args.cols && row0 + r0 + r < args.rows) at[r * args.ld] = t[r];
                }
              __syncwarp();
            }
          }
        }
      }
      ++ui;
    }
    if (!kSwap && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if constexpr (kCtas == 2) cluster_sync();  // nothing of either CTA is still signalled or read by the other
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    if constexpr (kCtas == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

template <typename T, int kFormat, int kN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Tile<kFormat, 2, kN>::kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_c,
                const __grid_constant__ CUtensorMap map_rs, const __grid_constant__ CUtensorMap map_cs,
                const __grid_constant__ CUtensorMap map_out, const Fp4TcArgs args, const Sched sc) {
  tc_body<T, kFormat, 2, kN, false>(map_r, map_c, map_rs, map_cs, map_out, args, sc);
}

template <typename T, int kFormat, int kN, bool kSwap>
__global__ void __launch_bounds__(Tile<kFormat, 1, kN>::kThreads, 1)
    single_kernel(const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_c,
                  const __grid_constant__ CUtensorMap map_rs, const __grid_constant__ CUtensorMap map_cs,
                  const __grid_constant__ CUtensorMap map_out, const Fp4TcArgs args, const Sched sc) {
  tc_body<T, kFormat, 1, kN, kSwap>(map_r, map_c, map_rs, map_cs, map_out, args, sc);
}

typedef void (*Kernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Fp4TcArgs, Sched);

struct Instance {
  Kernel kernel;
  size_t smem;
  int threads;
};

template <typename T, int kFormat>
Instance instance_t(Fp4TcShape shape) {
  auto single = [](auto* k, size_t smem, int threads) { return Instance{Kernel(k), smem, threads}; };
  using P = Tile<kFormat, 2, 256>;
  using Q = Tile<kFormat, 2, 128>;
  switch (shape) {
    case kFp4Pair256: return single(pair_kernel<T, kFormat, 256>, P::kSmem, P::kThreads);
    case kFp4Pair128: return single(pair_kernel<T, kFormat, 128>, Q::kSmem, Q::kThreads);
#define GB300_FP4_SINGLE(N, SWAP) \
  single(single_kernel<T, kFormat, N, SWAP>, Tile<kFormat, 1, N>::kSmem, Tile<kFormat, 1, N>::kThreads)
    case kFp4Single128: return GB300_FP4_SINGLE(128, false);
    case kFp4Swap16: return GB300_FP4_SINGLE(16, true);
    case kFp4Swap32: return GB300_FP4_SINGLE(32, true);
    case kFp4Swap64: return GB300_FP4_SINGLE(64, true);
#undef GB300_FP4_SINGLE
    default: return {};
  }
}

Instance instance(int dtype, int format, Fp4TcShape shape) {
  const bool mx = format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32: return mx ? instance_t<float, FP4_MXFP4>(shape) : instance_t<float, FP4_NVFP4>(shape);
    case FP4_BF16:
      return mx ? instance_t<__nv_bfloat16, FP4_MXFP4>(shape) : instance_t<__nv_bfloat16, FP4_NVFP4>(shape);
    default: return mx ? instance_t<__half, FP4_MXFP4>(shape) : instance_t<__half, FP4_NVFP4>(shape);
  }
}

}  // namespace

Fp4TcTile fp4_tc_tile(Fp4TcShape shape) {
  switch (shape) {
    case kFp4Pair256: return {256, 256, 2, false};
    case kFp4Pair128: return {256, 128, 2, false};
    case kFp4Single128: return {128, 128, 1, false};
    case kFp4Swap16: return {128, 16, 1, true};
    case kFp4Swap32: return {128, 32, 1, true};
    default: return {128, 64, 1, true};
  }
}

int fp4_tc_prepare() {
  int pairs = 0;
  for (int dtype = FP4_F32; dtype <= FP4_F16; ++dtype)
    for (int format = FP4_MXFP4; format <= FP4_NVFP4; ++format)
      for (int shape = 0; shape < kFp4TcShapes; ++shape) {
        const Instance in = instance(dtype, format, Fp4TcShape(shape));
        if (cudaFuncSetAttribute(reinterpret_cast<const void*>(in.kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 int(in.smem)) != cudaSuccess)
          return -1;
        if (fp4_tc_tile(Fp4TcShape(shape)).ctas == 2) {
          cudaLaunchConfig_t cfg = {};
          cfg.gridDim = dim3(2, 1, 1);
          cfg.blockDim = dim3(in.threads, 1, 1);
          cfg.dynamicSmemBytes = in.smem;
          int n = 0;
          if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(in.kernel), &cfg) != cudaSuccess) return -1;
          if (pairs == 0 || n < pairs) pairs = n;
        }
      }
  return pairs;
}

cudaError_t launch_fp4_tc(int dtype, int format, Fp4TcShape shape, const CUtensorMap (&maps)[5],
                          const Fp4TcArgs& args, const Sched& sc, int grid, cudaStream_t stream) {
  const Instance in = instance(dtype, format, shape);
  const int ctas = fp4_tc_tile(shape).ctas;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid * ctas), 1, 1);
  cfg.blockDim = dim3(unsigned(in.threads), 1, 1);
  cfg.dynamicSmemBytes = in.smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, in.kernel, maps[0], maps[1], maps[2], maps[3], maps[4], args, sc);
}

}  // namespace gb300
