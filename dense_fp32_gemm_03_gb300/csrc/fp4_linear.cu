// fp4_linear.cu -- the linear layer for up to 16 tokens in one kernel (fp4_linear
// in fp4.h): y = Q(x) W^T, x quantised on the way.
//
// Mathematics.  Q is fp4_quantize()'s, the product is fp4_gemm()'s; with this
// few rows of x the call is bound by reading W's codes and scales once, and
// below some tens of megabytes by its latencies.  So W's rows are the tensor
// core's 128 rows and the tokens its 16 columns, and K is split over the CTAs of a
// cluster: each quantises its part of x once, straight into the form that the tensor
// core reads, keeps it in shared memory and streams its part of one tile of W
// after another past it.  (A launch of its own for x would cost more than the whole of
// a small product.)  The cluster's sums meet in shared memory, sent by asynchronous
// stores that complete on the receiver's barrier: CTA r adds up and stores the r-th part
// of a tile's rows.
//
// Roles: warp 0 streams W, warp 1 issues the MMAs, warps 2 to 5 join and store,
// the others quantise x.
//
// What bounds it, measured.  1 x 4096 x 4096 (nvfp4, bf16; 9.4 MB) takes 5.4 to 6.4 us, of which
// the bytes are 1.4: launch, quantising x beside the first copies, one round to memory, the
// cluster's sum.  16 x 8192 x 8192 (mxfp4; 36 MB) takes 10.0 to 11.9 us, the bytes 5.3.
#include <cuda.h>
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "fp4_stream.cuh"
#include "sgemm_device.cuh"
#include "sgemm_internal.h"

namespace gb300 {
namespace {

using namespace fp4;

constexpr int kMaxQuantWarps = 16;
constexpr int kMaxThreads = 32 * (6 + kMaxQuantWarps);
constexpr int kCols = 16;       // tokens, the columns of a product
constexpr int kMaxSteps = 40;   // stages of K of one CTA
constexpr int kSumRow = kCols + 4;  // floats from one row's sums to the next: spreads the banks
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kStatusTimeout = 3;

// Shared memory: x (steps times codes and scales of 16 rows), the ring of W's
// stages, and the sums that the cluster's CTAs send (two tiles' worth).
template <int kFormat>
struct Layout {
  static constexpr uint32_t kWeights = Block<kFormat>::kBytes;
  static constexpr uint32_t kCodes = kCols * 128;
  static constexpr uint32_t kStep = kCodes + Block<kFormat>::kScales;
  static constexpr uint32_t kSums = 2 * 128 * kSumRow * 4;
  static constexpr uint32_t kArea = kSmemBytes - 1024 /* static */ - 1024 /* alignment */ - kSums;
  __host__ __device__ static constexpr uint32_t stages(uint32_t steps) {
    const uint32_t n = (kArea - steps * kStep) / kWeights;
    return n < uint32_t(kMaxStages) ? n : uint32_t(kMaxStages);
  }
  static_assert((kArea - kMaxSteps * kStep) / kWeights >= 2 && kStep % 1024 == 0 && kWeights % 1024 == 0, "shared memory");
};

struct Barriers {
  uint64_t full[kMaxStages], empty[kMaxStages], x[kMaxSteps], acc_full[2], acc_empty[2], sums[2], drain;
};

__device__ __forceinline__ uint32_t peer_address(const void* p, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(dev::smem_addr(p)), "r"(rank));
  return d;
}

// Waits for a barrier that other CTAs of the cluster arrive on, and sees what they wrote before.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint64_t limit, const volatile int* abort) {
  const uint64_t t0 = dev::global_timer_ns();
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(dev::smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if (*abort || dev::global_timer_ns() - t0 > limit) return false;
  }
}

// Sixteen consecutive values of a row as they are stored, zeros beyond `n`.
template <typename T>
struct Sixteen {
  static constexpr int kPieces = int(sizeof(T));  // of 16 bytes
  uint4 raw[kPieces];
  __device__ __forceinline__ void load(const T* row, int c, int n, bool vector) {
    if (vector && c + 16 <= n) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(row + c) + i);
    } else {
      T* t = reinterpret_cast<T*>(raw);
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = c + i < n ? row[c + i] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void values(float (&v)[16]) const {
    const T* t = reinterpret_cast<const T*>(raw);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = to_f32(t[i]);
  }
};

template <typename T, int kFormat>
__global__ void __launch_bounds__(kMaxThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map_w, const Fp4LinearArgs args) {
  using B = Block<kFormat>;
  using L = Layout<kFormat>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* area = smem_raw + ((1024u - (dev::smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ Barriers bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int ctas = args.ctas, cluster = blockIdx.x / ctas, clusters = gridDim.x / ctas, rank = blockIdx.x % ctas;
  const int tokens = args.tokens, tiles = (args.n + 127) / 128;
  // This CTA's stages of K.
  const int first = rank * args.per, steps = max(min(args.per, args.steps - first), 0);
  const uint32_t stages = L::stages(uint32_t(args.per));
  unsigned char* s_x = area;
  unsigned char* s_w = area + args.per * L::kStep;
  float* s_sums = reinterpret_cast<float*>(s_w + stages * L::kWeights);  // [tile parity][sender][own row][kSumRow]
  const int own = 128 / ctas;                                            // rows of a tile that a CTA adds up
  const uint64_t limit = args.wait_limit_ns;
  // A team of warps, two tokens to a warp, quantises one stage; teams take turns.
  const int team_warps = (tokens + 1) / 2, teams = (int(blockDim.x >> 5) - 6) / team_warps;

  auto load_stage = [&](int tile, int step, uint32_t slot) {
    unsigned char* stage = s_w + slot * L::kWeights;
    const uint32_t e = elected();
    expect_bytes(e, &bars.full[slot], L::kWeights);
    load_box<1>(e, stage, &map_w, (first + step) * 128, tile * 128, dev::smem_addr(&bars.full[slot]));
    load_bytes(e, stage + 16384, args.scales + (int64_t(tile) * args.steps + first + step) * B::kScales, B::kScales,
               &bars.full[slot]);
  };
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dev::smem_addr(&s_tmem)),
                 "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {
    if (lane < kMaxStages) {
      dev::mbar_init(&bars.full[lane], 1);
      dev::mbar_init(&bars.empty[lane], 1);
    }
    for (int i = lane; i < steps; i += 32) dev::mbar_init(&bars.x[i], uint32_t(team_warps));
    if (lane < 2) {
      dev::mbar_init(&bars.acc_full[lane], 1);
      dev::mbar_init(&bars.acc_empty[lane], 4);
      dev::mbar_init(&bars.sums[lane], 1);
    }
    if (lane == 2) {
      dev::mbar_init(&bars.drain, 1);
      s_abort = 0;
    }
    dev::mbar_init_fence();
    __syncwarp();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // The ring's first stages need no other warp: they go out before the CTA's barrier.
    for (uint32_t n = 0; n < stages && int(n) < steps; ++n) {
      load_stage(cluster, int(n), n);
    }
  }
  // The kernel before on the stream may still run up to here (16 x 8192 x 8192, one call after
  // another: 12.3 us launched in order, 10.0 so).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // So do the first values of x.
  const int team = (warp - 6) / team_warps, token = (warp - 6) % team_warps * 2 + (lane >> 4), chunk = lane & 15;
  const bool quantises = warp >= 6 && warp - 6 < teams * team_warps, in = quantises && token < tokens;
  const T* x_row = static_cast<const T*>(args.x) + int64_t(in ? token : 0) * args.ldx;
  const bool vector = (reinterpret_cast<uintptr_t>(args.x) & 15u) == 0 && args.ldx % int64_t(16 / sizeof(T)) == 0;
  // Every CTA reads the same lines of x at about the same time, which makes each
  // read take 2000 cycles or so: kAhead of them are under way.
  constexpr int kAhead = sizeof(T) == 4 ? 2 : 3;
  Sixteen<T> x_values[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = team + j * teams;
    if (in && i < steps) x_values[j].load(x_row, (first + i) * 256 + chunk * 16, args.k, vector);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (ctas > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  constexpr uint32_t tmem = kTmemBase;
  auto fail = [&]() {
    if (!s_abort) {
      s_abort = 1;
      dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
    }
  };
  // The other CTAs' barriers exist once this has been waited for (before the first signal).
  auto wait_started = [&]() {
    if (ctas > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };

  if (warp == 0) {
    // ---- W: codes (TMA, 128-byte swizzle) and scale atoms (one contiguous piece)
    wait_started();
    At put;
    bool go = true;
    for (int tile = cluster; go && tile < tiles; tile += clusters)
      for (int i = 0; i < steps; ++i, put.next(stages)) {
        if (tile == cluster && i < int(stages)) continue;  // on its way
        if (put.lap > 0 && !dev::mbar_wait_abortable(&bars.empty[put.slot], (put.lap - 1) & 1u, limit, &s_abort)) fail();
        go = __shfl_sync(kFull, s_abort, 0) == 0;
        if (!go) break;
        load_stage(tile, i, put.slot);
      }
  } else if (warp == 1) {
    // ---- MMAs
    wait_started();
    At got;
    uint32_t done = 0;
    for (int tile = cluster; tile < tiles; tile += clusters, ++done) {
      const uint32_t b = done & 1u, nb = done >> 1;
      if (nb > 0 && !dev::mbar_wait_abortable(&bars.acc_empty[b], (nb - 1) & 1u, limit, &s_abort)) fail();
      for (int i = 0; i < steps; ++i) {
        if (done == 0 && !dev::mbar_wait_abortable(&bars.x[i], 0u, limit, &s_abort)) fail();
        if (!dev::mbar_wait_abortable(&bars.full[got.slot], got.lap & 1u, limit, &s_abort)) fail();
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t e = elected();
        const uint32_t base = dev::smem_addr(s_w + got.slot * L::kWeights), xs = dev::smem_addr(s_x + i * L::kStep);
        const uint32_t sr = tmem + 256 + got.slot * (8 * B::kAtoms), sc = sr + 4 * B::kAtoms;
        const uint64_t drs = scale_desc(base + 16384), dcs = scale_desc(xs + L::kCodes);
#pragma unroll
        for (int a = 0; a < B::kAtoms; ++a) {
          copy_scales<1>(e, sr + 4 * a, drs + 32 * a);
          copy_scales<1>(e, sc + 4 * a, dcs + 32 * a);
        }
        const uint64_t dr = operand_desc(base), dc = operand_desc(xs);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          constexpr int kPer = 4 / B::kAtoms;  // MMAs that share an atom
          const int a = j / kPer;
          mma<kFormat, 1>(e, tmem + b * kCols, dr + 2 * j, dc + 2 * j,
                          instr_desc<kFormat>(128, kCols, kPer == 2 ? (j & 1) * 2 : 0), sr + 4 * a, sc + 4 * a,
                          (i != 0 || j != 0) ? 1u : 0u);
        }
        commit<1>(e, &bars.empty[got.slot]);
        got.next(stages);
      }
      commit<1>(elected(), &bars.acc_full[b]);
    }
    commit<1>(elected(), &bars.drain);
    dev::mbar_wait(&bars.drain, 0u, limit);
  } else if (warp < 6) {
    // ---- joining and storing: a lane has one row of W, 16 tokens
    const int q = warp & 3, row_local = 32 * q + lane;
    float2 alpha = make_float2(1.f, 1.f);
    if (kFormat == FP4_NVFP4)
      alpha = join_factors(args.w_factor ? __ldg(args.w_factor) : 1.f, args.x_factor ? __ldg(args.x_factor) : 1.f);
    T* y = static_cast<T*>(args.y);
    wait_started();
    uint32_t done = 0;
    for (int tile = cluster; tile < tiles; tile += clusters, ++done) {
      const uint32_t b = done & 1u, nb = done >> 1;
      if (!dev::mbar_wait_abortable(&bars.acc_full[b], nb & 1u, limit, &s_abort)) fail();
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      __syncwarp();
      float sum[kCols];
      {
        uint32_t* r = reinterpret_cast<uint32_t*>(sum);
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
              "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(tmem + b * kCols + (uint32_t(32 * q) << 16)));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      }
      if (steps == 0) {  // K has fewer stages than the cluster has CTAs
#pragma unroll
        for (int t = 0; t < kCols; ++t) sum[t] = 0.f;
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) dev::mbar_arrive(&bars.acc_empty[b]);
      const int row = tile * 128 + row_local;
      if (ctas == 1) {
        if (row < args.n) {
#pragma unroll
          for (int t = 0; t < kCols; ++t)
            if (t < tokens) y[int64_t(t) * args.ldy + row] = from_f32<T>(sum[t] * alpha.x * alpha.y);
        }
        continue;
      }
      // Each row's sums to the CTA that adds them up.  A buffer is free again once the tile
      // after it was joined: a CTA's warps send that tile's rows only when all are through with this one.
      if (done > 0) dev::named_barrier(1, 128);
      float* mine = s_sums + b * (128 * kSumRow);
      const int vectors = (tokens + 3) / 4;
      if (warp == 2 && lane == 0) dev::mbar_arrive_expect_tx(&bars.sums[b], uint32_t(128 * vectors * 16));
      const uint32_t to = peer_address(mine + (rank * own + row_local % own) * kSumRow, uint32_t(row_local / own));
      const uint32_t bar = peer_address(&bars.sums[b], uint32_t(row_local / own));
#pragma unroll
      for (int t = 0; t < kCols; t += 4)
        if (t < tokens)
          asm volatile(
              "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                  to + t * 4),
              "r"(__float_as_uint(sum[t])), "r"(__float_as_uint(sum[t + 1])), "r"(__float_as_uint(sum[t + 2])),
              "r"(__float_as_uint(sum[t + 3])), "r"(bar)
              : "memory");
      if (!wait_cluster(&bars.sums[b], nb & 1u, limit, &s_abort)) fail();
      const int own_row = (threadIdx.x - 64) % own, out_row = tile * 128 + rank * own + own_row;
      if (out_row < args.n) {
        for (int t = (threadIdx.x - 64) / own; t < tokens; t += ctas) {
          const float* p = mine + own_row * kSumRow + t;
          float total = p[0];
          for (int c = 1; c < ctas; ++c) total += p[c * own * kSumRow];
          y[int64_t(t) * args.ldy + out_row] = from_f32<T>(total * alpha.x * alpha.y);
        }
      }
      __syncwarp();
    }
  } else {
    // ---- x: 16 lanes to a token, 16 values of K to a lane
    if (quantises) {
      const Quantizer<kFormat> quantizer(args.x_factor);
      for (int i0 = team; i0 < steps; i0 += kAhead * teams) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int i = i0 + j * teams;
          if (i >= steps) break;
          float v[16];
          x_values[j].values(v);
          const int next = i + kAhead * teams;
          if (in && next < steps) x_values[j].load(x_row, (first + next) * 256 + chunk * 16, args.k, vector);
          float a = largest(v), unit;
          if (Format<kFormat>::kBlock == 32) a = max_abs(a, __shfl_xor_sync(kFull, a, 1));
          const uint32_t byte = quantizer.scale(a, unit);
          uint32_t word[2];
          quantizer.encode(v, a, unit, word);
          if (in) {
            unsigned char* columns = s_x + i * L::kStep;
            *reinterpret_cast<uint2*>(columns + piece_at(uint32_t(token), uint32_t(chunk >> 1)) + (chunk & 1) * 8) =
                make_uint2(word[0], word[1]);
            constexpr int kPer = Format<kFormat>::kBlock / 16;  // lanes of a block
            if (chunk % kPer == 0) columns[L::kCodes + scale_at(uint32_t(token), uint32_t(chunk / kPer))] = uint8_t(byte);
          }
          dev::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) dev::mbar_arrive(&bars.x[i]);
        }
      }
    }
    wait_started();
  }
  __syncwarp();
  if (s_abort && threadIdx.x == 0) {
    // Copies still under way get a bounded time to land before the CTA's memory goes.
    const uint64_t t0 = dev::global_timer_ns();
    while (dev::global_timer_ns() - t0 < 100000ull) __nanosleep(1000);
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (ctas > 1)  // nothing of this CTA is still written by another
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

struct Instance {
  const void* kernel;
  size_t smem;
};

template <typename T>
Instance instance_t(int format) {
  return format == FP4_MXFP4
             ? Instance{reinterpret_cast<const void*>(&linear_kernel<T, FP4_MXFP4>), size_t(kSmemBytes) - 1024}
             : Instance{reinterpret_cast<const void*>(&linear_kernel<T, FP4_NVFP4>), size_t(kSmemBytes) - 1024};
}

Instance instance(int dtype, int format) {
  return dtype == FP4_F32 ? instance_t<float>(format)
         : dtype == FP4_BF16 ? instance_t<__nv_bfloat16>(format)
                             : instance_t<__half>(format);
}

cudaLaunchConfig_t config(const Instance& in, int clusters, int ctas, int quant_warps, cudaLaunchAttribute (&attributes)[2]) {
  attributes[0].id = cudaLaunchAttributeClusterDimension;
  attributes[0].val.clusterDim.x = unsigned(ctas);
  attributes[0].val.clusterDim.y = 1;
  attributes[0].val.clusterDim.z = 1;
  attributes[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attributes[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(clusters * ctas), 1, 1);
  cfg.blockDim = dim3(unsigned(32 * (6 + quant_warps)), 1, 1);
  cfg.dynamicSmemBytes = in.smem;
  cfg.attrs = attributes;
  cfg.numAttrs = 2;
  return cfg;
}

}  // namespace

int fp4_linear_tokens() { return kCols; }
int fp4_linear_steps() { return kMaxSteps; }

bool fp4_linear_prepare(int (&clusters)[4]) {
  for (int i = 0; i < 4; ++i) clusters[i] = 0;
  for (int dtype = FP4_F32; dtype <= FP4_F16; ++dtype)
    for (int format = FP4_MXFP4; format <= FP4_NVFP4; ++format) {
      const Instance in = instance(dtype, format);
      if (cudaFuncSetAttribute(in.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(in.smem)) != cudaSuccess)
        return false;
      for (int i = 0; i < 4; ++i) {
        cudaLaunchAttribute attributes[2] = {};
        const cudaLaunchConfig_t cfg = config(in, 1, 1 << i, kMaxQuantWarps, attributes);
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, in.kernel, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        if (clusters[i] == 0 || n < clusters[i]) clusters[i] = n;
      }
    }
  return true;
}

cudaError_t launch_fp4_linear(int dtype, int format, const CUtensorMap& map, const Fp4LinearArgs& args, int clusters,
                              cudaStream_t stream) {
  const Instance in = instance(dtype, format);
  cudaLaunchAttribute attributes[2] = {};
  // As many teams as there are stages to quantise, up to the most warps: idle warps only delay the start.
  const int team_warps = (args.tokens + 1) / 2, wanted = team_warps * args.per;
  cudaLaunchConfig_t cfg =
      config(in, clusters, args.ctas, wanted < kMaxQuantWarps ? wanted : kMaxQuantWarps, attributes);
  cfg.stream = stream;
  CUtensorMap m = map;
  Fp4LinearArgs a = args;
  void* params[] = {&m, &a};
  return cudaLaunchKernelExC(&cfg, in.kernel, params);
}

}  // namespace gb300
