// fp4_moe.cu -- the mixture-of-experts layer on 4-bit weights for a few
// tokens (fp4_moe in fp4.h), and the order of its weights.
//
// Mathematics.  A token takes part in `top` of the experts, so a few tokens
// touch each expert's weights for one or two columns only: the layer is bound
// by reading the weights once.  Weights become 16-bit floats (exact) in
// registers and are multiplied by mma.m16n8k16, 16 weight rows by eight
// columns.  Activations enter as 16-bit floats relative to a power of two of
// the token: one column a token where x has 16 bits, two (the value rounded
// to 11 bits, and the rest) where it has 32.  A block's products are summed
// first and then scaled by its unit, in 32 bits.
#include <cuda_runtime.h>

#include "fp4_device.cuh"
#include "fp4_internal.h"
#include "sgemm_device.cuh"

namespace gb300 {
namespace {

using namespace fp4;

constexpr int kPackThreads = 256;
constexpr int kThreads = 512;  // of the layer's kernel, one CTA to an SM
constexpr int kWarps = kThreads / 32;
constexpr int kTeamWarps = 4;  // warps that share a gate-and-up tile
constexpr int kTeams = kWarps / kTeamWarps;
constexpr int kRing = 4;  // chunks that a warp has under way
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTop = 32;
constexpr int kMaxPairs = kMoeTokens * kMaxTop;
constexpr int kMaxParts = 8;
constexpr uint32_t kStatusTimeout = 3;

template <int kFormat>
struct Chunk {  // 16 rows x 128 columns
  static constexpr int kScaleBytes = 16 * 128 / Format<kFormat>::kBlock;
  static constexpr int kBytes = 1024 + kScaleBytes;
};

// ------------------------------------------------------------------ packing
// One thread makes the 16 bytes of one lane and half of a chunk.  Row g and
// row g + 8 of a gate-and-up tile are gate row 8 tile + g and up row 8 tile + g.
template <int kFormat, bool kGateUp>
__global__ void __launch_bounds__(kPackThreads)
    pack_experts_kernel(const fp4_matrix_t q, int64_t experts, int64_t rows_per, uint8_t* __restrict__ out) {
  using F = Format<kFormat>;
  const int64_t tiles = kGateUp ? (rows_per + 7) / 8 : (rows_per + 15) / 16;
  const int64_t chunks = (q.cols + 127) / 128;
  const int64_t atoms = (q.cols + 255) / 256 * F::kAtomsPerStage;
  const int64_t items = experts * tiles * chunks * 64;
  for (int64_t i = int64_t(blockIdx.x) * kPackThreads + threadIdx.x; i < items;
       i += int64_t(gridDim.x) * kPackThreads) {
    const int lane = int(i & 31), half = int(i >> 5) & 1;
    const int64_t c = (i >> 6) % chunks, tile = (i >> 6) / chunks % tiles, e = (i >> 6) / chunks / tiles;
    const int g = lane >> 2, t = lane & 3;
    int64_t row[2];
    bool in[2];
    if (kGateUp) {
      const int64_t r = tile * 8 + g;
      in[0] = in[1] = r < rows_per;
      row[0] = e * 2 * rows_per + r;
      row[1] = row[0] + rows_per;
    } else {
      for (int s = 0; s < 2; ++s) {
        const int64_t r = tile * 16 + g + 8 * s;
        in[s] = r < rows_per;
        row[s] = e * rows_per + r;
      }
    }
    uint8_t* dst = out + ((e * tiles + tile) * chunks + c) * Chunk<kFormat>::kBytes;
    uint32_t word[4];
    for (int j = 0; j < 4; ++j) {
      const int64_t k = c * 128 + half * 64 + j * 16 + t * 4;
      uint32_t v[2];
      for (int s = 0; s < 2; ++s)
        v[s] = in[s] && k < q.cols ? *reinterpret_cast<const uint16_t*>(q.codes + row[s] * q.ld + k / 2) : 0u;
      word[j] = (v[0] & 0xffu) | (v[1] & 0xffu) << 8 | (v[0] >> 8) << 16 | (v[1] >> 8) << 24;
    }
    reinterpret_cast<uint4*>(dst)[half * 32 + lane] = make_uint4(word[0], word[1], word[2], word[3]);
    // Scales of row pair g: the blocks of row g, then those of row g + 8.
    constexpr int kPer = 128 / F::kBlock;
    if (half == 0 && t < 2) {
      for (int b = 0; b < kPer; ++b) {
        const int64_t k = c * kPer + b;
        dst[1024 + g * 2 * kPer + t * kPer + b] =
            in[t] && k * F::kBlock < q.cols ? q.scales[scale_offset(row[t], k, atoms)] : 0;
      }
    }
  }
}

// ------------------------------------------------------------------ helpers
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint2 b) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// The power of two that brings a largest magnitude (as bits) to [2^14, 2^15),
// well inside a 16-bit float; at most 2^126, and 1 for 0, NaN and infinity.
__device__ __forceinline__ float pow2_scale(uint32_t top) {
  if (top == 0 || top >= 0x7f800000u) return 1.f;
  const int e = int(top >> 23);  // 127 + floor(log2)
  return __uint_as_float(uint32_t(min(127 + 14 + 127 - e, 253)) << 23);
}

// Column of the mma: token and part.  kSplit: columns 2 n and 2 n + 1 are the
// rounded value and the rest of token n.
template <bool kSplit>
struct Columns {
  static constexpr int kTokens = kSplit ? 4 : 8;  // per group of eight columns
  __device__ static int token(int group, int col) { return group * kTokens + (kSplit ? col >> 1 : col); }
};

// Four values (times `scale`) as the two B registers of this lane.
template <bool kSplit>
__device__ __forceinline__ uint2 to_frag(const float4& v, float scale, int col) {
  const float x[4] = {v.x * scale, v.y * scale, v.z * scale, v.w * scale};
  __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
  if (kSplit && (col & 1)) {
    const float2 fa = __half22float2(a), fb = __half22float2(b);
    a = __floats2half2_rn(x[0] - fa.x, x[1] - fa.y);
    b = __floats2half2_rn(x[2] - fb.x, x[3] - fb.y);
  }
  return make_uint2(h2_bits(a), h2_bits(b));
}

// A chunk of weights on its way through registers: codes of 64 columns each,
// and the scale bytes of row g (first half) and row g + 8.
template <int kFormat>
struct ChunkRegs {
  static constexpr int kPer = 128 / Format<kFormat>::kBlock;  // blocks of a row
  uint4 w[2];
  uint32_t sc[2][kPer / 4];

  __device__ __forceinline__ void load(const uint8_t* __restrict__ chunk, int lane) {
    const uint4* codes = reinterpret_cast<const uint4*>(chunk);
    w[0] = __ldg(codes + lane);
    w[1] = __ldg(codes + 32 + lane);
    if constexpr (kPer == 8) {
      const uint4 s = __ldg(reinterpret_cast<const uint4*>(chunk + 1024) + (lane >> 2));
      sc[0][0] = s.x, sc[0][1] = s.y, sc[1][0] = s.z, sc[1][1] = s.w;
    } else {
      const uint2 s = __ldg(reinterpret_cast<const uint2*>(chunk + 1024) + (lane >> 2));
      sc[0][0] = s.x, sc[1][0] = s.y;
    }
  }
};

// acc[q] += (16 rows x 128 columns of weights) * (128 x 8 columns of group q),
// for the groups in `mask`.  frag(q, s) gives the lane's B registers of the
// steps 2 s and 2 s + 1.
template <int kFormat, int kGroups, typename Frag>
__device__ __forceinline__ void chunk_mma(const ChunkRegs<kFormat>& in, uint32_t mask, float (&acc)[kGroups][4],
                                          Frag frag) {
  constexpr int kSteps = Format<kFormat>::kBlock / 16;  // mma steps of a block
#pragma unroll
  for (int p = 0; p < 4; ++p) {  // two steps, 32 columns
    uint32_t a[2][4];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int step = 2 * p + s;
      const uint4& h = in.w[step >> 2];
      const uint32_t word = (step & 3) == 0 ? h.x : (step & 3) == 1 ? h.y : (step & 3) == 2 ? h.z : h.w;
      a[s][0] = h2_bits(decode2<0>(word));
      a[s][1] = h2_bits(decode2<1>(word));
      a[s][2] = h2_bits(decode2<2>(word));
      a[s][3] = h2_bits(decode2<3>(word));
    }
    float u[2][2 / kSteps];  // units: row g or g + 8, block
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int s = 0; s < 2 / kSteps; ++s) {
        const int b = p * (2 / kSteps) + s;
        u[r][s] = decode_scale<kFormat>((in.sc[r][b / 4] >> (8 * (b & 3))) & 0xffu);
      }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (kGroups > 1 && !(mask >> q & 1)) continue;
      const uint4 f = frag(q, p);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma16816(d, a[0][0], a[0][1], a[0][2], a[0][3], make_uint2(f.x, f.y));
      if constexpr (kSteps == 1) {
        acc[q][0] = fmaf(u[0][0], d[0], acc[q][0]);
        acc[q][1] = fmaf(u[0][0], d[1], acc[q][1]);
        acc[q][2] = fmaf(u[1][0], d[2], acc[q][2]);
        acc[q][3] = fmaf(u[1][0], d[3], acc[q][3]);
        d[0] = d[1] = d[2] = d[3] = 0.f;
      }
      mma16816(d, a[1][0], a[1][1], a[1][2], a[1][3], make_uint2(f.z, f.w));
      constexpr int kLast = 2 / kSteps - 1;
      acc[q][0] = fmaf(u[0][kLast], d[0], acc[q][0]);
      acc[q][1] = fmaf(u[0][kLast], d[1], acc[q][1]);
      acc[q][2] = fmaf(u[1][kLast], d[2], acc[q][2]);
      acc[q][3] = fmaf(u[1][kLast], d[3], acc[q][3]);
    }
  }
}

// Sum over `warps` warps' accumulators of (row, token): red is [warp][group][4][32].
template <bool kSplit, int kGroups>
__device__ __forceinline__ float reduce(const float* red, int warps, int row, int token) {
  const int q = token / Columns<kSplit>::kTokens, n = token % Columns<kSplit>::kTokens;
  const int g = row & 7, upper = (row >> 3) * 2;
  float sum = 0.f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    const float* p = red + (w * kGroups + q) * 128;
    if (kSplit)
      sum += p[upper * 32 + g * 4 + n] + p[(upper + 1) * 32 + g * 4 + n];
    else
      sum += p[(upper + (n & 1)) * 32 + g * 4 + (n >> 1)];
  }
  return sum;
}

template <int kGroups>
__device__ __forceinline__ void publish(float* red, const float (&acc)[kGroups][4], int warp, int lane) {
#pragma unroll
  for (int q = 0; q < kGroups; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((warp * kGroups + q) * 4 + i) * 32 + lane] = acc[q][i];
}

// ------------------------------------------------------------------ routing
// Order of logits as integers: larger first; NaN last, below every number.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x7fffffffu) > 0x7f800000u ? 1u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp: the `top` largest of one token's logits (equal ones by index) and
// their softmax weights.  A lane keeps the logits of its experts in registers.
template <int kPerLane>
__device__ __forceinline__ void select_top(const float* logits, int experts, int top, int renorm, int lane,
                                           uint16_t* ids, float* weight) {
  float v[kPerLane];
  uint32_t key[kPerLane];
  float peak = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < experts ? __ldcg(logits + e) : -INFINITY;
    key[i] = e < experts ? order_key(v[i]) : 0u;
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) peak = fmaxf(peak, v[i]);
  for (int s = 16; s; s >>= 1) peak = fmaxf(peak, __shfl_xor_sync(kFull, peak, s));
#pragma unroll
  for (int i = 0; i < kPerLane; ++i)
    if (lane + 32 * i < experts) sum += expf(v[i] - peak);
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
  float mine = 0.f;
  int mine_id = 0;
  for (int j = 0; j < top; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) best = max(best, key[i]);
    const uint32_t peak_key = __reduce_max_sync(kFull, best);
    int at = kMaxExperts;
#pragma unroll
    for (int i = kPerLane - 1; i >= 0; --i)
      if (key[i] == peak_key) at = lane + 32 * i;
    const int id = int(__reduce_min_sync(kFull, unsigned(at)));
    float p = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 32 * i == id) {
        key[i] = 0;
        p = expf(v[i] - peak) / sum;
      }
    p = __shfl_sync(kFull, p, id & 31);
    if (lane == j) mine = p, mine_id = id;
  }
  if (renorm) {
    float total = mine;
    for (int s = 16; s; s >>= 1) total += __shfl_xor_sync(kFull, total, s);
    mine /= total;
  }
  if (lane < top) {
    ids[lane] = uint16_t(mine_id);
    weight[lane] = mine;
  }
}

// Four consecutive values of a row, zeros beyond `n`.
template <typename T>
__device__ __forceinline__ float4 load4(const T* p, int k, int n, bool vector) {
  if (vector && k + 4 <= n) {
    if constexpr (sizeof(T) == 4) {
      return __ldg(reinterpret_cast<const float4*>(p + k));
    } else {
      const uint2 r = __ldg(reinterpret_cast<const uint2*>(p + k));
      const T* t = reinterpret_cast<const T*>(&r);
      return make_float4(to_f32(t[0]), to_f32(t[1]), to_f32(t[2]), to_f32(t[3]));
    }
  }
  float4 v;
  v.x = k < n ? to_f32(p[k]) : 0.f;
  v.y = k + 1 < n ? to_f32(p[k + 1]) : 0.f;
  v.z = k + 2 < n ? to_f32(p[k + 2]) : 0.f;
  v.w = k + 3 < n ? to_f32(p[k + 3]) : 0.f;
  return v;
}

// ------------------------------------------------------------- grid barrier
// All CTAs are resident (cooperative launch).  Every thread returns the same
// answer: false once the bounded wait ran out.
__device__ __forceinline__ bool grid_barrier(int32_t* counter, const MoeArgs& args, int* s_ok) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1);
    int ok = 1;
    const uint64_t t0 = dev::global_timer_ns();
    while (dev::ld_acquire_gpu(counter) < int(gridDim.x)) {
      if (dev::global_timer_ns() - t0 > args.wait_limit_ns) {
        dev::record_status(args.status, kStatusTimeout, kWaitTileStage);
        ok = 0;
        break;
      }
    }
    __threadfence();
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0;
}

// -------------------------------------------------------------------- layer
// Three phases with a grid barrier between them.
//  1. Router: a CTA to an expert computes the logits of all tokens; a CTA to a
//     token makes its fragments.
//  2. Every CTA selects the experts (the same way), then teams of four warps
//     compute gate-and-up tiles (8 values of h), K shared among the warps.
//  3. The CTA's 16 warps share the K of all experts in use for one tile of 16
//     rows of y; where whole tiles leave SMs idle, a tile's experts are cut into
//     `parts`, joined in order by the last CTA to finish one.
// Weights stream through a ring of four chunks a warp, across tile borders.
template <typename T, int kFormat, bool kSplitX, int kGroupsX, bool kSplitH, int kGroupsH>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const MoeArgs args) {
  constexpr int kRedX = kTeams * kTeamWarps * kGroupsX * 128, kRedH = kWarps * kGroupsH * 128;
  __shared__ float s_red[kRedX > kRedH ? kRedX : kRedH];
  __shared__ float s_weight[kMoeTokens][kMaxTop];
  __shared__ uint16_t s_ids[kMoeTokens][kMaxTop];
  __shared__ uint16_t s_mask[kMaxExperts];        // tokens that go to an expert
  __shared__ uint16_t s_active[kMaxPairs];        // experts in use, in order
  __shared__ uint8_t s_slot[kMaxPairs][kMoeTokens];  // place of an expert in use among a token's
  __shared__ int s_count, s_flag;
  __shared__ uint32_t s_top;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tokens = args.tokens, experts = args.experts, top = args.top, d = args.d, f = args.f;
  const int d_chunks = (d + 127) / 128, f_chunks = (f + 127) / 128;

  // ---- router and fragments
  {
    const T* x = static_cast<const T*>(args.x);
    const bool vec_x = (reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T))) == 0 && args.ldx % 4 == 0;
    const bool vec_r = (reinterpret_cast<uintptr_t>(args.router) & 15u) == 0 && args.ldr % 4 == 0;
    const int share = kWarps / tokens;  // warps to a token
    for (int item = blockIdx.x; item < experts + tokens; item += gridDim.x) {
      if (item < experts) {
        const float* r = args.router + item * args.ldr;
        float sum = 0.f;
        const int t = warp / share, part = warp % share;
        if (t < tokens) {
          const T* xt = x + t * args.ldx;
#pragma unroll 4
          for (int k = (part * 32 + lane) * 4; k < d; k += share * 128) {
            const float4 a = load4(xt, k, d, vec_x), b = load4(r, k, d, vec_r);
            sum = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, sum))));
          }
          for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
          if (lane == 0) s_red[warp] = sum;
        }
        __syncthreads();
        if (threadIdx.x < tokens) {
          float total = 0.f;
          for (int w = 0; w < share; ++w) total += s_red[threadIdx.x * share + w];
          args.logits[threadIdx.x * experts + item] = total;
        }
        __syncthreads();
      } else {
        const int t = item - experts;
        const T* xt = x + t * args.ldx;
        if (threadIdx.x == 0) s_top = 0;
        __syncthreads();
        uint32_t most = 0;
        for (int k = threadIdx.x * 4; k < d; k += kThreads * 4) {
          const float4 v = load4(xt, k, d, vec_x);
          most = max(max(max(most, __float_as_uint(v.x) & 0x7fffffffu), __float_as_uint(v.y) & 0x7fffffffu),
                     max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
        }
        most = __reduce_max_sync(kFull, most);
        if (lane == 0) atomicMax(&s_top, most);
        __syncthreads();
        const float scale = pow2_scale(s_top);
        const int group = t / Columns<kSplitX>::kTokens, n = t % Columns<kSplitX>::kTokens;
        // Fragments: steps 2 s and 2 s + 1 of a lane (column, l) lie together.
        uint2* frag = static_cast<uint2*>(args.x_frag) + int64_t(group) * d_chunks * 256;
        for (int i = threadIdx.x; i < d_chunks * 32; i += kThreads) {
          const float4 v = load4(xt, i * 4, d, vec_x);
          const int step = i >> 2, l = i & 3;
#pragma unroll
          for (int part = 0; part < (kSplitX ? 2 : 1); ++part) {
            const int col = kSplitX ? 2 * n + part : n;
            frag[((step >> 1) * 32 + col * 4 + l) * 2 + (step & 1)] = to_frag<kSplitX>(v, scale, col);
          }
        }
        if (threadIdx.x == 0) {
          args.x_scale[t] = scale;
          args.h_max[t] = 0;
        }
        __syncthreads();
      }
    }
  }
  if (!grid_barrier(args.counters, args, &s_flag)) return;

  // ---- selection, the same in every CTA
  for (int e = threadIdx.x; e < experts; e += kThreads) s_mask[e] = 0;
  if (warp < tokens) {
    const float* l = args.logits + warp * experts;
    if (experts <= 64)
      select_top<2>(l, experts, top, args.renormalize, lane, s_ids[warp], s_weight[warp]);
    else if (experts <= 256)
      select_top<8>(l, experts, top, args.renormalize, lane, s_ids[warp], s_weight[warp]);
    else
      select_top<32>(l, experts, top, args.renormalize, lane, s_ids[warp], s_weight[warp]);
    __syncwarp();
    if (blockIdx.x == 0 && lane < top) {
      if (args.ids) args.ids[warp * top + lane] = s_ids[warp][lane];
      if (args.p) args.p[warp * top + lane] = s_weight[warp][lane];
    }
  }
  __syncthreads();
  if (warp == 0) {
    // Masks token by token (a token's experts differ), then the experts in use in order.
    for (int t = 0; t < tokens; ++t) {
      if (lane < top) s_mask[s_ids[t][lane]] |= uint16_t(1u << t);
      __syncwarp();
    }
    int count = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + lane;
      const bool in = e < experts && s_mask[e] != 0;
      const uint32_t vote = __ballot_sync(kFull, in);
      if (in) s_active[count + __popc(vote & ((1u << lane) - 1u))] = uint16_t(e);
      count += __popc(vote);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int used = s_count;
  for (int i = threadIdx.x; i < used * tokens; i += kThreads) {
    const int a = i / tokens, t = i - a * tokens, e = s_active[a];
    int slot = 255;
    if (s_mask[e] >> t & 1)
      for (int j = 0; j < top; ++j)
        if (s_ids[t][j] == e) slot = j;
    s_slot[a][t] = uint8_t(slot);
  }
  __syncthreads();

  // ---- gate and up
  {
    const int team = warp / kTeamWarps, member = warp % kTeamWarps, tid = threadIdx.x % (32 * kTeamWarps);
    const int tiles = (f + 7) / 8, total = used * tiles, stride = int(gridDim.x) * kTeams;
    const int rounds = (d_chunks + kTeamWarps - 1) / kTeamWarps;  // chunks of a warp and tile
    float* red = s_red + team * (kTeamWarps * kGroupsX * 128);
    const uint4* frags = static_cast<const uint4*>(args.x_frag);
    const float factor = args.gate_up_factor ? __ldg(args.gate_up_factor) : 1.f;
    ChunkRegs<kFormat> ring[kRing];
    // Neighbouring teams take neighbouring CTAs' tiles, so that a last, partial
    // round spreads over the SMs.
    int load_unit = team * int(gridDim.x) + int(blockIdx.x), load_i = 0, unit = load_unit, i = 0;
    const uint8_t* load_base = nullptr;
    auto locate = [&]() {
      if (load_unit < total) {
        const int a = load_unit / tiles;
        load_base = args.gate_up + (int64_t(s_active[a]) * tiles + (load_unit - a * tiles)) * d_chunks * Chunk<kFormat>::kBytes;
      }
    };
    auto load_next = [&](ChunkRegs<kFormat>& r) {
      const int c = load_i * kTeamWarps + member;
      if (load_unit < total && c < d_chunks) r.load(load_base + int64_t(c) * Chunk<kFormat>::kBytes, lane);
      if (++load_i == rounds) {
        load_i = 0;
        load_unit += stride;
        locate();
      }
    };
    locate();
#pragma unroll
    for (int s = 0; s < kRing; ++s) load_next(ring[s]);
    float acc[kGroupsX][4] = {};
    int a = unit < total ? unit / tiles : 0;
    auto groups_of = [&](int active) {
      uint32_t m = 0;
      if (unit < total) {
        const uint32_t t = s_mask[s_active[active]];
#pragma unroll
        for (int q = 0; q < kGroupsX; ++q)
          if (t >> (q * Columns<kSplitX>::kTokens) & ((1u << Columns<kSplitX>::kTokens) - 1u)) m |= 1u << q;
      }
      return m;
    };
    uint32_t mask = groups_of(a);
    while (unit < total) {
#pragma unroll
      for (int s = 0; s < kRing; ++s) {
        if (unit < total) {
          const int c = i * kTeamWarps + member;
          if (c < d_chunks)
            chunk_mma<kFormat, kGroupsX>(ring[s], mask, acc,
                                         [&](int q, int p) { return frags[(int64_t(q) * d_chunks + c) * 128 + p * 32 + lane]; });
          load_next(ring[s]);
          if (++i == rounds) {
            publish<kGroupsX>(red, acc, member, lane);
            dev::named_barrier(1 + team, 32 * kTeamWarps);
            const int t = tid >> 3, r = tid & 7, slot = t < tokens ? s_slot[a][t] : 255;
            if (slot != 255) {
              const float u = factor / args.x_scale[t];
              const float gate = reduce<kSplitX, kGroupsX>(red, kTeamWarps, r, t) * u;
              const float up = reduce<kSplitX, kGroupsX>(red, kTeamWarps, r + 8, t) * u;
              const float h = gate / (1.f + expf(-gate)) * up * s_weight[t][slot];
              args.h[int64_t(t * top + slot) * f_chunks * 128 + (unit - a * tiles) * 8 + r] = h;
              atomicMax(args.h_max + t, __float_as_uint(h) & 0x7fffffffu);
            }
            dev::named_barrier(1 + team, 32 * kTeamWarps);
#pragma unroll
            for (int q = 0; q < kGroupsX; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
            i = 0;
            unit += stride;
            a = unit < total ? unit / tiles : 0;
            mask = groups_of(a);
          }
        }
      }
    }
  }
  if (!grid_barrier(args.counters + 1, args, &s_flag)) return;

  // ---- down
  {
    const int tiles = (d + 15) / 16, f8 = (f + 7) / 8 * 8, list = used * f_chunks, ctas = int(gridDim.x);
    // Parts of a tile: the fewest that keep the CTAs within a few percent of the
    // best balance, with two chunks a warp at least.
    int parts = 1;
    {
      float best = float((tiles + ctas - 1) / ctas);
      for (int p = 2; p <= kMaxParts && list / p >= 2 * kWarps && tiles <= args.tile_counter_count; ++p) {
        const float cost = float((tiles * p + ctas - 1) / ctas) / float(p);
        if (cost < 0.95f * best) best = cost, parts = p;
      }
    }
    const int total = tiles * parts, per = (list + parts - 1) / parts;
    const float factor = args.down_factor ? __ldg(args.down_factor) : 1.f;
    const int col = lane >> 2;
    float scale[kGroupsH];
    int token[kGroupsH];
#pragma unroll
    for (int q = 0; q < kGroupsH; ++q) {
      token[q] = Columns<kSplitH>::token(q, col);
      scale[q] = token[q] < tokens ? pow2_scale(__ldcg(args.h_max + token[q])) : 0.f;
    }
    ChunkRegs<kFormat> ring[kRing];
    int load_unit = blockIdx.x, load_at = 0, load_end = 0, unit = blockIdx.x, at = 0, end = 0;
    auto span = [&](int u, int& begin, int& stop) {
      const int p = u % parts;
      begin = min(p * per, list);
      stop = min(begin + per, list);
    };
    auto load_next = [&](ChunkRegs<kFormat>& r) {
      if (load_unit < total) {
        const int l = load_at + warp;
        if (l < load_end) {
          const int e = l / f_chunks, c = l - e * f_chunks;
          r.load(args.down + ((int64_t(s_active[e]) * tiles + load_unit / parts) * f_chunks + c) * Chunk<kFormat>::kBytes,
                 lane);
        }
        load_at += kWarps;
        if (load_at >= load_end) {
          load_unit += ctas;
          span(load_unit, load_at, load_end);
        }
      }
    };
    span(load_unit, load_at, load_end);
    span(unit, at, end);
#pragma unroll
    for (int s = 0; s < kRing; ++s) load_next(ring[s]);
    float acc[kGroupsH][4] = {};
    while (unit < total) {
#pragma unroll
      for (int s = 0; s < kRing; ++s) {
        if (unit < total) {
          const int l = at + warp;
          if (l < end) {
            const int e = l / f_chunks, c = l - e * f_chunks;
            const float* rows[kGroupsH];
            uint32_t mask = 0;
#pragma unroll
            for (int q = 0; q < kGroupsH; ++q) {
              const int slot = token[q] < tokens ? s_slot[e][token[q]] : 255;
              rows[q] = slot != 255 ? args.h + int64_t(token[q] * top + slot) * f_chunks * 128 : nullptr;
              if (__any_sync(kFull, slot != 255)) mask |= 1u << q;
            }
            chunk_mma<kFormat, kGroupsH>(ring[s], mask, acc, [&](int q, int p) {
              uint2 b[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int k = c * 128 + (2 * p + j) * 16 + (lane & 3) * 4;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (rows[q] != nullptr && k < f8) v = *reinterpret_cast<const float4*>(rows[q] + k);
                b[j] = to_frag<kSplitH>(v, scale[q], col);
              }
              return make_uint4(b[0].x, b[0].y, b[1].x, b[1].y);
            });
          }
          load_next(ring[s]);
          at += kWarps;
          if (at >= end) {
            const int tile = unit / parts, part = unit - tile * parts;
            publish<kGroupsH>(s_red, acc, warp, lane);
            __syncthreads();
            const int t = threadIdx.x >> 4, r = threadIdx.x & 15, row = tile * 16 + r;
            const bool mine = t < tokens;  // threads beyond 16 tokens: none
            float y = 0.f;
            if (mine) y = reduce<kSplitH, kGroupsH>(s_red, kWarps, r, t);
            bool store = true;
            if (parts > 1) {
              float* share = args.partial + int64_t(tile) * parts * (16 * kMoeTokens);
              if (mine) __stcg(share + part * (16 * kMoeTokens) + t * 16 + r, y);
              __syncthreads();
              if (threadIdx.x == 0) {
                __threadfence();
                s_flag = atomicAdd(args.tile_counters + tile, 1) == parts - 1;
                __threadfence();
              }
              __syncthreads();
              store = s_flag != 0;
              if (store) {
                if (mine) {
                  y = 0.f;
                  for (int p = 0; p < parts; ++p) y += __ldcg(share + p * (16 * kMoeTokens) + t * 16 + r);
                }
                if (threadIdx.x == 0) args.tile_counters[tile] = 0;
              }
            }
            if (store && mine && row < d)
              static_cast<T*>(args.y)[t * args.ldy + row] =
                  from_f32<T>(y * (factor / pow2_scale(__ldcg(args.h_max + t))));
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kGroupsH; ++q) acc[q][0] = acc[q][1] = acc[q][2] = acc[q][3] = 0.f;
            unit += ctas;
            span(unit, at, end);
          }
        }
      }
    }
  }
  // The last CTA to leave clears the barriers' counters for the next call.
  if (threadIdx.x == 0 && atomicAdd(args.counters + 2, 1) == int(gridDim.x) - 1) {
    args.counters[0] = 0;
    args.counters[1] = 0;
    args.counters[2] = 0;
  }
}

template <typename T, int kFormat, bool kSplitX, int kGroupsX, bool kSplitH, int kGroupsH>
cudaError_t launch_t(const MoeArgs& args, int sms, cudaStream_t stream) {
  MoeArgs copy = args;
  void* params[] = {&copy};
  return cudaLaunchCooperativeKernel(
      reinterpret_cast<const void*>(&moe_kernel<T, kFormat, kSplitX, kGroupsX, kSplitH, kGroupsH>), dim3(unsigned(sms)),
      dim3(kThreads), params, 0, stream);
}

// Columns of eight that the tokens take, for x and for h: a 32-bit x and its h
// are split in two; h beside a 16-bit float x too, since one rounding to its 11
// bits would show in the result; bfloat16 has 8.
template <int kFormat>
cudaError_t launch_format(int dtype, const MoeArgs& args, int sms, cudaStream_t stream) {
  const int t = args.tokens;
  switch (dtype) {
    case FP4_F32:
      if (t <= 4) return launch_t<float, kFormat, true, 1, true, 1>(args, sms, stream);
      if (t <= 8) return launch_t<float, kFormat, true, 2, true, 2>(args, sms, stream);
      return launch_t<float, kFormat, true, 4, true, 4>(args, sms, stream);
    case FP4_BF16:
      if (t <= 8) return launch_t<__nv_bfloat16, kFormat, false, 1, false, 1>(args, sms, stream);
      return launch_t<__nv_bfloat16, kFormat, false, 2, false, 2>(args, sms, stream);
    default:
      if (t <= 4) return launch_t<__half, kFormat, false, 1, true, 1>(args, sms, stream);
      if (t <= 8) return launch_t<__half, kFormat, false, 1, true, 2>(args, sms, stream);
      return launch_t<__half, kFormat, false, 2, true, 4>(args, sms, stream);
  }
}

size_t round_up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

int64_t fp4_expert_chunk_bytes(int format) {
  return format == FP4_MXFP4 ? Chunk<FP4_MXFP4>::kBytes : Chunk<FP4_NVFP4>::kBytes;
}

MoeScratch fp4_moe_scratch(int dtype, int64_t tokens, int64_t experts, int64_t d, int64_t f, int64_t top) {
  MoeScratch s{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round_up(bytes);
    return here;
  };
  const int64_t per = dtype == FP4_F32 ? 4 : 8;
  s.logits = take(tokens * experts * 4);
  s.x_scale = take(tokens * 4);
  s.h_max = take(tokens * 4);
  s.x_frag = take((tokens + per - 1) / per * ((d + 127) / 128) * 8 * 32 * 8);
  s.h = take(tokens * top * ((f + 127) / 128) * 128 * 4);
  s.partial = take(((d + 15) / 16) * kMaxParts * 16 * kMoeTokens * 4);
  s.bytes = at;
  return s;
}

cudaError_t launch_fp4_experts_pack(const fp4_matrix_t& gate_up, const fp4_matrix_t& down,
                                    const fp4_experts_t& w, cudaStream_t stream) {
  auto grid = [](int64_t items) {
    const int64_t b = (items + kPackThreads - 1) / kPackThreads;
    return unsigned(b < (1 << 20) ? b : (1 << 20));
  };
  const int64_t up_items = w.experts * ((w.f + 7) / 8) * ((w.d + 127) / 128) * 64;
  const int64_t down_items = w.experts * ((w.d + 15) / 16) * ((w.f + 127) / 128) * 64;
  if (w.format == FP4_MXFP4) {
    pack_experts_kernel<FP4_MXFP4, true><<<grid(up_items), kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up);
    pack_experts_kernel<FP4_MXFP4, false><<<grid(down_items), kPackThreads, 0, stream>>>(down, w.experts, w.d, w.down);
  } else {
    pack_experts_kernel<FP4_NVFP4, true><<<grid(up_items), kPackThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up);
    pack_experts_kernel<FP4_NVFP4, false><<<grid(down_items), kPackThreads, 0, stream>>>(down, w.experts, w.d, w.down);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int sms, cudaStream_t stream) {
  return format == FP4_MXFP4 ? launch_format<FP4_MXFP4>(dtype, args, sms, stream)
                             : launch_format<FP4_NVFP4>(dtype, args, sms, stream);
}

}  // namespace gb300
