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

namespace gb300 {
namespace {

using namespace fp4;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxExperts = 1024;

template <int kFormat>
struct Chunk {  // 16 rows x 128 columns
  static constexpr int kScaleBytes = 16 * 128 / Format<kFormat>::kBlock;
  static constexpr int kBytes = 1024 + kScaleBytes;
};

// ------------------------------------------------------------------ packing
// One thread makes the 16 bytes of one lane and half of a chunk.  Row g and
// row g + 8 of a gate-and-up tile are gate row 8 tile + g and up row 8 tile + g.
template <int kFormat, bool kGateUp>
__global__ void __launch_bounds__(kThreads)
    pack_experts_kernel(const fp4_matrix_t q, int64_t experts, int64_t rows_per, uint8_t* __restrict__ out) {
  using F = Format<kFormat>;
  const int64_t tiles = kGateUp ? (rows_per + 7) / 8 : (rows_per + 15) / 16;
  const int64_t chunks = (q.cols + 127) / 128;
  const int64_t atoms = (q.cols + 255) / 256 * F::kAtomsPerStage;
  const int64_t items = experts * tiles * chunks * 64;
  for (int64_t i = int64_t(blockIdx.x) * kThreads + threadIdx.x; i < items; i += int64_t(gridDim.x) * kThreads) {
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

// acc[q] += (16 rows x 128 columns of weights) * (128 x 8 columns of group q),
// for the groups in `mask`.  frag(q, s) is the lane's B registers of step s.
template <int kFormat, int kGroups, typename Frag>
__device__ __forceinline__ void chunk_mma(const uint8_t* __restrict__ chunk, int lane, uint32_t mask,
                                          float (&acc)[kGroups][4], Frag frag) {
  const uint4* codes = reinterpret_cast<const uint4*>(chunk);
  uint4 w[2] = {__ldg(codes + lane), __ldg(codes + 32 + lane)};
  constexpr int kPer = 128 / Format<kFormat>::kBlock;  // blocks of a row
  uint32_t sc[2][kPer / 4];
  if constexpr (kPer == 8) {
    const uint4 s = __ldg(reinterpret_cast<const uint4*>(chunk + 1024) + (lane >> 2));
    sc[0][0] = s.x, sc[0][1] = s.y, sc[1][0] = s.z, sc[1][1] = s.w;
  } else {
    const uint2 s = __ldg(reinterpret_cast<const uint2*>(chunk + 1024) + (lane >> 2));
    sc[0][0] = s.x, sc[1][0] = s.y;
  }
  constexpr int kSteps = Format<kFormat>::kBlock / 16;  // mma steps of a block
#pragma unroll
  for (int b = 0; b < kPer; ++b) {
    const float u0 = decode_scale<kFormat>((sc[0][b / 4] >> (8 * (b & 3))) & 0xffu);
    const float u1 = decode_scale<kFormat>((sc[1][b / 4] >> (8 * (b & 3))) & 0xffu);
    uint32_t a[kSteps][4];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int step = b * kSteps + s;
      const uint4& h = w[step >> 2];
      const uint32_t word = (step & 3) == 0 ? h.x : (step & 3) == 1 ? h.y : (step & 3) == 2 ? h.z : h.w;
      a[s][0] = h2_bits(decode2<0>(word));
      a[s][1] = h2_bits(decode2<1>(word));
      a[s][2] = h2_bits(decode2<2>(word));
      a[s][3] = h2_bits(decode2<3>(word));
    }
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (!(mask >> q & 1)) continue;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) mma16816(d, a[s][0], a[s][1], a[s][2], a[s][3], frag(q, b * kSteps + s));
      acc[q][0] = fmaf(u0, d[0], acc[q][0]);
      acc[q][1] = fmaf(u0, d[1], acc[q][1]);
      acc[q][2] = fmaf(u1, d[2], acc[q][2]);
      acc[q][3] = fmaf(u1, d[3], acc[q][3]);
    }
  }
}

// Sum over the warps' accumulators of (row g or g + 8, token n): red is [warp][group][4][32].
template <bool kSplit, int kGroups>
__device__ __forceinline__ float reduce(const float* red, int row, int token) {
  const int q = token / Columns<kSplit>::kTokens, n = token % Columns<kSplit>::kTokens;
  const int g = row & 7, upper = (row >> 3) * 2;
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
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
// Order of logits: larger first, equal ones by index; NaN last.
__device__ __forceinline__ uint64_t order_key(float v, int index) {
  uint32_t b = __float_as_uint(v + 0.f);
  b = (b & 0x7fffffffu) > 0x7f800000u ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
  return uint64_t(b) << 32 | (0xffffffffu - uint32_t(index));
}

// One warp: the `top` largest of one token's logits, their softmax weights.
__device__ __forceinline__ void select_top(const float* logits, int experts, int top, int renorm, int lane,
                                           int32_t* ids, float* weight) {
  float peak = -INFINITY, sum = 0.f;
  for (int e = lane; e < experts; e += 32) peak = fmaxf(peak, __ldcg(logits + e));
  for (int s = 16; s; s >>= 1) peak = fmaxf(peak, __shfl_xor_sync(kFull, peak, s));
  for (int e = lane; e < experts; e += 32) sum += expf(__ldcg(logits + e) - peak);
  for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
  uint64_t last = ~0ull;
  float mine = 0.f, total = 0.f;
  int mine_id = 0;
  for (int j = 0; j < top; ++j) {
    uint64_t best = 0;
    for (int e = lane; e < experts; e += 32) {
      const uint64_t k = order_key(__ldcg(logits + e), e);
      if (k < last && k > best) best = k;
    }
    for (int s = 16; s; s >>= 1) {
      const uint64_t o = __shfl_xor_sync(kFull, best, s);
      best = o > best ? o : best;
    }
    last = best;
    const int id = int(0xffffffffu - uint32_t(best));
    const float p = expf(__ldcg(logits + id) - peak) / sum;
    total += p;
    if (lane == j) mine = p, mine_id = id;
  }
  if (lane < top) {
    ids[lane] = mine_id;
    weight[lane] = renorm ? mine / total : mine;
  }
}

template <typename T, bool kSplit>
__global__ void __launch_bounds__(kThreads) route_kernel(const MoeArgs args) {
  __shared__ uint32_t s_top;
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(args.x) + t * args.ldx;
  if (threadIdx.x == 0) s_top = 0;
  __syncthreads();
  for (int e = warp; e < args.experts; e += kWarps) {
    const float* r = args.router + e * args.ldr;
    float sum = 0.f;
    for (int k = lane; k < args.d; k += 32) sum = fmaf(to_f32(x[k]), r[k], sum);
    for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(kFull, sum, s);
    if (lane == 0) args.logits[t * args.experts + e] = sum;
  }
  uint32_t top = 0;
  for (int k = threadIdx.x; k < args.d; k += kThreads) top = max(top, __float_as_uint(to_f32(x[k])) & 0x7fffffffu);
  atomicMax(&s_top, top);
  __syncthreads();
  const float scale = pow2_scale(s_top);
  // Fragments: step s, lane (column g, t): values 16 s + 4 t .. + 3.
  const int steps = (args.d + 127) / 128 * 8;
  const int group = t / Columns<kSplit>::kTokens, n = t % Columns<kSplit>::kTokens;
  uint2* frag = static_cast<uint2*>(args.x_frag) + int64_t(group) * steps * 32;
  for (int i = threadIdx.x; i < steps * 4; i += kThreads) {
    const int k = i * 4;
    float4 v;
    v.x = k < args.d ? to_f32(x[k]) : 0.f;
    v.y = k + 1 < args.d ? to_f32(x[k + 1]) : 0.f;
    v.z = k + 2 < args.d ? to_f32(x[k + 2]) : 0.f;
    v.w = k + 3 < args.d ? to_f32(x[k + 3]) : 0.f;
    for (int part = 0; part < (kSplit ? 2 : 1); ++part) {
      const int col = kSplit ? 2 * n + part : n;
      frag[(i >> 2) * 32 + col * 4 + (i & 3)] = to_frag<kSplit>(v, scale, col);
    }
  }
  if (threadIdx.x == 0) {
    args.x_scale[t] = scale;
    args.h_max[t] = 0;
  }
  if (warp == 0) {
    select_top(args.logits + t * args.experts, args.experts, args.top, args.renormalize, lane,
               args.pick + t * args.top, args.weight + t * args.top);
    __syncwarp();
    if (lane < args.top) {
      if (args.ids) args.ids[t * args.top + lane] = args.pick[t * args.top + lane];
      if (args.p) args.p[t * args.top + lane] = args.weight[t * args.top + lane];
    }
  }
}

// ------------------------------------------------------------- gate and up
template <int kFormat, bool kSplit, int kGroups>
__global__ void __launch_bounds__(kThreads) up_kernel(const MoeArgs args) {
  __shared__ float red[kWarps * kGroups * 128];
  __shared__ int s_slot[kMoeTokens];
  const int e = blockIdx.y, tile = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kMoeTokens) {
    int slot = -1;
    if (threadIdx.x < args.tokens)
      for (int j = 0; j < args.top; ++j)
        if (args.pick[threadIdx.x * args.top + j] == e) slot = j;
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();
  uint32_t mask = 0;
  for (int t = 0; t < args.tokens; ++t)
    if (s_slot[t] >= 0) mask |= 1u << (t / Columns<kSplit>::kTokens);
  if (mask == 0) return;
  const int chunks = (args.d + 127) / 128, steps = chunks * 8, tiles = (args.f + 7) / 8;
  const uint2* frags = static_cast<const uint2*>(args.x_frag);
  float acc[kGroups][4] = {};
  for (int c = warp; c < chunks; c += kWarps)
    chunk_mma<kFormat, kGroups>(
        args.gate_up + ((int64_t(e) * tiles + tile) * chunks + c) * Chunk<kFormat>::kBytes, lane, mask, acc,
        [&](int q, int s) { return frags[(int64_t(q) * steps + c * 8 + s) * 32 + lane]; });
  publish<kGroups>(red, acc, warp, lane);
  __syncthreads();
  const int t = threadIdx.x >> 3, r = threadIdx.x & 7;
  if (t < args.tokens && s_slot[t] >= 0) {
    const float u = (args.gate_up_factor ? *args.gate_up_factor : 1.f) / args.x_scale[t];
    const float gate = reduce<kSplit, kGroups>(red, r, t) * u, up = reduce<kSplit, kGroups>(red, r + 8, t) * u;
    const int pair = t * args.top + s_slot[t];
    const float h = gate / (1.f + expf(-gate)) * up * args.weight[pair];
    args.h[int64_t(pair) * ((args.f + 127) / 128 * 128) + tile * 8 + r] = h;
    atomicMax(args.h_max + t, __float_as_uint(h) & 0x7fffffffu);
  }
}

// --------------------------------------------------------------------- down
template <typename T, int kFormat, bool kSplit, int kGroups>
__global__ void __launch_bounds__(kThreads) down_kernel(const MoeArgs args) {
  __shared__ float red[kWarps * kGroups * 128];
  const int tile = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (args.f + 127) / 128, tiles = (args.d + 15) / 16, f8 = (args.f + 7) / 8 * 8;
  const int col = lane >> 2;
  float acc[kGroups][4] = {};
  float scale[kGroups];
  for (int q = 0; q < kGroups; ++q) {
    const int t = Columns<kSplit>::token(q, col);
    scale[q] = t < args.tokens ? pow2_scale(args.h_max[t]) : 0.f;
  }
  for (int e = 0; e < args.experts; ++e) {
    uint32_t mask = 0;
    const float* rows[kGroups];
    for (int q = 0; q < kGroups; ++q) {
      const int t = Columns<kSplit>::token(q, col);
      rows[q] = nullptr;
      if (t < args.tokens)
        for (int j = 0; j < args.top; ++j)
          if (args.pick[t * args.top + j] == e) rows[q] = args.h + int64_t(t * args.top + j) * chunks * 128;
      if (__any_sync(kFull, rows[q] != nullptr)) mask |= 1u << q;
    }
    if (mask == 0) continue;
    for (int c = warp; c < chunks; c += kWarps)
      chunk_mma<kFormat, kGroups>(
          args.down + ((int64_t(e) * tiles + tile) * chunks + c) * Chunk<kFormat>::kBytes, lane, mask, acc,
          [&](int q, int s) {
            const int k = c * 128 + s * 16 + (lane & 3) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (rows[q] != nullptr && k < f8) v = *reinterpret_cast<const float4*>(rows[q] + k);
            return to_frag<kSplit>(v, scale[q], col);
          });
  }
  publish<kGroups>(red, acc, warp, lane);
  __syncthreads();
  const int t = threadIdx.x >> 4, r = threadIdx.x & 15, row = tile * 16 + r;
  if (t < args.tokens && row < args.d) {
    const float u = (args.down_factor ? *args.down_factor : 1.f) / pow2_scale(args.h_max[t]);
    static_cast<T*>(args.y)[t * args.ldy + row] = from_f32<T>(reduce<kSplit, kGroups>(red, r, t) * u);
  }
}

template <typename T, int kFormat, bool kSplit, int kGroups>
cudaError_t launch_t(const MoeArgs& args, cudaStream_t stream) {
  route_kernel<T, kSplit><<<args.tokens, kThreads, 0, stream>>>(args);
  up_kernel<kFormat, kSplit, kGroups><<<dim3((args.f + 7) / 8, args.experts), kThreads, 0, stream>>>(args);
  down_kernel<T, kFormat, kSplit, kGroups><<<(args.d + 15) / 16, kThreads, 0, stream>>>(args);
  return cudaGetLastError();
}

template <typename T, int kFormat, bool kSplit>
cudaError_t launch_groups(const MoeArgs& args, cudaStream_t stream) {
  const int groups = (args.tokens + Columns<kSplit>::kTokens - 1) / Columns<kSplit>::kTokens;
  if (groups <= 1) return launch_t<T, kFormat, kSplit, 1>(args, stream);
  if (groups <= 2) return launch_t<T, kFormat, kSplit, 2>(args, stream);
  if constexpr (kSplit) return launch_t<T, kFormat, kSplit, 4>(args, stream);
  return cudaErrorInvalidValue;
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
  s.pick = take(tokens * top * 4);
  s.weight = take(tokens * top * 4);
  s.x_scale = take(tokens * 4);
  s.h_max = take(tokens * 4);
  s.x_frag = take((tokens + per - 1) / per * ((d + 127) / 128) * 8 * 32 * 8);
  s.h = take(tokens * top * ((f + 127) / 128) * 128 * 4);
  s.bytes = at;
  return s;
}

cudaError_t launch_fp4_experts_pack(const fp4_matrix_t& gate_up, const fp4_matrix_t& down,
                                    const fp4_experts_t& w, cudaStream_t stream) {
  auto grid = [](int64_t items) {
    const int64_t b = (items + kThreads - 1) / kThreads;
    return unsigned(b < (1 << 20) ? b : (1 << 20));
  };
  const int64_t up_items = w.experts * ((w.f + 7) / 8) * ((w.d + 127) / 128) * 64;
  const int64_t down_items = w.experts * ((w.d + 15) / 16) * ((w.f + 127) / 128) * 64;
  if (w.format == FP4_MXFP4) {
    pack_experts_kernel<FP4_MXFP4, true><<<grid(up_items), kThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up);
    pack_experts_kernel<FP4_MXFP4, false><<<grid(down_items), kThreads, 0, stream>>>(down, w.experts, w.d, w.down);
  } else {
    pack_experts_kernel<FP4_NVFP4, true><<<grid(up_items), kThreads, 0, stream>>>(gate_up, w.experts, w.f, w.gate_up);
    pack_experts_kernel<FP4_NVFP4, false><<<grid(down_items), kThreads, 0, stream>>>(down, w.experts, w.d, w.down);
  }
  return cudaGetLastError();
}

cudaError_t launch_fp4_moe(int dtype, int format, const MoeArgs& args, int /*sms*/, cudaStream_t stream) {
  const bool mx = format == FP4_MXFP4;
  switch (dtype) {
    case FP4_F32:
      return mx ? launch_groups<float, FP4_MXFP4, true>(args, stream)
                : launch_groups<float, FP4_NVFP4, true>(args, stream);
    case FP4_BF16:
      return mx ? launch_groups<__nv_bfloat16, FP4_MXFP4, false>(args, stream)
                : launch_groups<__nv_bfloat16, FP4_NVFP4, false>(args, stream);
    default:
      return mx ? launch_groups<__half, FP4_MXFP4, false>(args, stream)
                : launch_groups<__half, FP4_NVFP4, false>(args, stream);
  }
}

}  // namespace gb300
