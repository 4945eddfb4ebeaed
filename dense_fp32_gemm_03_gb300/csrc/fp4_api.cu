// fp4_api.cu -- host side of the 4-bit operators' C ABI (include/fp4.h):
// argument validation, scratch and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <array>
#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>

#include "fp4.h"
#include "fp4_internal.h"
#include "sgemm_internal.h"

namespace {

using gb300::LibDevice;

// Rows and columns: tile and piece counts stay within 32 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 30;

int64_t block_of(int format) { return format == FP4_MXFP4 ? 32 : 16; }
int64_t dtype_bytes(int dtype) { return dtype == FP4_F32 ? 4 : 2; }
int64_t code_pitch(int64_t cols) { return (cols + 31) / 32 * 16; }
int64_t scale_bytes(int format, int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * ((cols + 255) / 256) * (64 / block_of(format)) * 512;
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

sgemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

sgemm_status_t check_format(int format) {
  return format == FP4_MXFP4 || format == FP4_NVFP4 ? SGEMM_OK : SGEMM_ERR_INVALID_VALUE;
}

sgemm_status_t check_extent(int64_t a, int64_t b) {
  if (a < 0 || b < 0) return SGEMM_ERR_INVALID_VALUE;
  return a > kMaxExtent || b > kMaxExtent ? SGEMM_ERR_UNSUPPORTED : SGEMM_OK;
}

sgemm_status_t check_quantized(const fp4_matrix_t* q) {
  if (q == nullptr || check_format(q->format) != SGEMM_OK) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(q->rows, q->cols);
  if (st != SGEMM_OK) return st;
  if (q->rows == 0 || q->cols == 0) return SGEMM_OK;
  if (q->codes == nullptr || q->scales == nullptr || !aligned(q->codes, 16) || !aligned(q->scales, 16) ||
      q->ld < code_pitch(q->cols) || q->ld % 16 != 0 || !aligned(q->factor, 4))
    return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

// An unquantised rows x cols matrix.
sgemm_status_t check_dense(int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (dtype < FP4_F32 || dtype > FP4_F16) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(rows, cols);
  if (st != SGEMM_OK) return st;
  if (rows == 0 || cols == 0) return SGEMM_OK;
  if (p == nullptr || ld < cols || !aligned(p, size_t(dtype_bytes(dtype)))) return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

struct Range {
  uintptr_t lo, hi;
};
Range range(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, bytes > 0 ? a + uintptr_t(bytes) : a};
}
Range dense_range(int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return range(p, rows && cols ? ((rows - 1) * ld + cols) * dtype_bytes(dtype) : 0);
}
Range code_range(const fp4_matrix_t* q) {
  return range(q->codes, q->rows && q->cols ? (q->rows - 1) * q->ld + code_pitch(q->cols) : 0);
}
Range scale_range(const fp4_matrix_t* q) { return range(q->scales, scale_bytes(q->format, q->rows, q->cols)); }
Range factor_range(const float* f) { return range(f, f ? 4 : 0); }
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool overlap(Range a, const fp4_matrix_t* q) {
  return overlap(a, code_range(q)) || overlap(a, scale_range(q)) || overlap(a, factor_range(q->factor));
}

// ------------------------------------------------------------------- products
std::mutex g_mu;
std::map<int, int> g_pairs;  // CTA pairs that run at once, by device

// The experts' kernels, prepared once a device.
std::map<int, bool> g_moe;

bool moe_ready(int dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = g_moe.find(dev);
  if (it == g_moe.end()) it = g_moe.emplace(dev, gb300::fp4_moe_prepare()).first;
  return it->second;
}

int tc_pairs(int dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = g_pairs.find(dev);
  if (it == g_pairs.end()) it = g_pairs.emplace(dev, gb300::fp4_tc_prepare()).first;
  return it->second;
}

struct Product {
  gb300::Fp4TcShape shape;
  gb300::Sched sc;
  int grid;
  size_t partial_bytes;
  double us;  // estimated time, launch aside
};

// Times (us), fitted to GB300 timings from 512 x 512 x 8192 to 8192^3: a 256-column
// step of K of one tile; what a tile adds to its steps; storing a tile of 32-bit
// outputs, beside the next tile's steps or after the last; what a launch of pairs
// adds; joining tiles that are split over K, beyond the steps that it saves (1024 x
// 1024 x 16384: 17.9 us split, 16.1 us whole; 20 x 8192 x 8192: 13.0 and 10.8; pairs of
// CTAs, 4096^3: 50 and 35, so pairs never split).  One CTA adds up a tile's shares, one
// after another (100 x 128 x 40000 in 152: 118 us).
struct ShapeCost {
  double step, tile, store, launch, join, share;
};
ShapeCost shape_cost(gb300::Fp4TcShape s) {
  switch (s) {
    case gb300::kFp4Pair256: return {0.36, 0.9, 3.4, 0.6, 0.0, 0.0};
    case gb300::kFp4Pair128: return {0.205, 0.4, 2.6, 0.6, 0.0, 0.0};
    case gb300::kFp4Single128: return {0.225, 0.4, 2.5, 0.0, 9.0, 0.7};
    default: return {0.2, 0.3, 0.0, 0.0, 6.0, 0.25};
  }
}

// Stores of 16-bit outputs, and of rows that TMA does not reach (4096 x 4097 x 1024:
// 34.8 us in 32 bits, 4096 x 4096 x 1024: 19.6; in 16 bits 22.9 and 16.8).
double store_cost(bool bytes4, bool tma) { return tma ? (bytes4 ? 1.0 : 0.85) : (bytes4 ? 2.35 : 1.35); }

bool stores_by_tma(const void* C, int64_t ldc, int64_t cols, int64_t es) {
  return aligned(C, 16) && ldc * es % 16 == 0 && cols * es < (int64_t(1) << 31);
}

// Tiles go to `units` CTAs (pairs) in waves.  If that is estimated to be faster, those of
// the last, partial wave are cut over K in equal shares, one to a unit, but no more
// than balance the steps that a share saves with what adding it costs.
bool plan_tiles(int64_t rows, int64_t cols, int64_t K, gb300::Fp4TcShape shape, int units, double stores,
                Product* p) {
  const gb300::Fp4TcTile t = gb300::fp4_tc_tile(shape);
  const int64_t tm = (rows + t.rows - 1) / t.rows, tn = (cols + t.cols - 1) / t.cols, tiles = tm * tn;
  if (tiles > 0x7fffffffLL || units <= 0) return false;
  const ShapeCost c = shape_cost(shape);
  const int64_t steps = (K + 255) / 256, waves = (tiles + units - 1) / units, rest = tiles % units;
  p->shape = shape;
  p->sc = gb300::Sched{};
  p->sc.tiles_m = int32_t(tm);
  p->sc.tiles_n = int32_t(tn);
  p->sc.group_m = gb300::kGroupM;
  p->sc.iters_per_tile = int32_t(steps);
  p->sc.dp_tiles = int32_t(tiles);
  p->grid = int(tiles < units ? tiles : units);
  p->partial_bytes = 0;
  const double store = stores * c.store, whole = std::max(double(steps) * c.step + c.tile, store);
  p->us = double(waves) * whole + store + c.launch;
  const int64_t total = rest * steps;
  if (t.ctas != 1 || rest == 0 || rest > int64_t(gb300::kWorkspaceCounterBytes / 4)) return true;
  const double balance = std::sqrt(double(steps) * c.step / c.share);
  int64_t shares = int64_t(balance) * rest;
  if (shares > units) shares = units;
  if (shares > total) shares = total;
  if (shares <= rest) return true;
  const double split_us = double(waves - 1) * whole + double((total + shares - 1) / shares) * c.step + c.tile + store +
                          c.join +
                          double(shares) / double(rest) * c.share;
  if (split_us >= p->us) return true;
  p->us = split_us;
  p->sc.dp_tiles = int32_t(tiles - rest);
  p->sc.sk_tiles = int32_t(rest);
  p->sc.sk_ctas = int32_t(shares);
  p->sc.sk_base = int32_t(total / shares);
  p->sc.sk_extra = int32_t(total % shares);
  p->grid = p->sc.dp_tiles > 0 ? units : int(shares);
  p->partial_bytes = size_t(rest + shares - 1) * t.rows * t.cols * 4;
  return true;
}

// Few rows of A: B supplies the tile rows and A the columns, as few as hold
// them.  Otherwise the tiles that are estimated to be fastest: pairs of CTAs share what
// they read, 256 columns more of it than 128 (8192^3: 166 us, 128 columns 177, single
// CTAs 213), and smaller tiles fill the last wave better (4096^3: 32.0, 29.2, 32.3) or
// the only one (1024^3: 7.1, 6.0, 5.2).
bool plan_product(int64_t M, int64_t N, int64_t K, int sms, int pairs, int64_t es, const void* C, int64_t ldc,
                  Product* p) {
  if (M <= 64) {
    const gb300::Fp4TcShape s = M <= 16 ? gb300::kFp4Swap16 : M <= 32 ? gb300::kFp4Swap32 : gb300::kFp4Swap64;
    return plan_tiles(N, M, K, s, sms, 0.0, p);
  }
  const double stores = store_cost(es == 4, stores_by_tma(C, ldc, N, es));
  bool any = false;
  for (const gb300::Fp4TcShape s : {gb300::kFp4Pair256, gb300::kFp4Pair128, gb300::kFp4Single128}) {
    Product q{};
    if (!plan_tiles(M, N, K, s, s == gb300::kFp4Single128 ? sms : pairs, stores, &q)) continue;
    if (!any || q.us < p->us) *p = q;
    any = true;
  }
  return any;
}

// The linear layer for few tokens: K over the CTAs of a cluster, a tile of 128
// rows of W to a cluster at a time.  The cluster size with the fewest stages one
// after another in a CTA; the smallest such, since joining costs.
struct Clusters {
  int ctas, clusters;
  int64_t steps, per;
};
std::map<int, std::array<int, 4>> g_clusters;  // of 1, 2, 4 and 8 CTAs that run at once, by device

bool plan_linear(int64_t M, int64_t N, int64_t K, int dev, Clusters* c) {
  if (M > gb300::fp4_linear_tokens()) return false;
  std::array<int, 4> most;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    auto it = g_clusters.find(dev);
    if (it == g_clusters.end()) {
      int n[4];
      if (!gb300::fp4_linear_prepare(n)) n[0] = n[1] = n[2] = n[3] = 0;
      it = g_clusters.emplace(dev, std::array<int, 4>{n[0], n[1], n[2], n[3]}).first;
    }
    most = it->second;
  }
  const int64_t tiles = (N + 127) / 128, steps = (K + 255) / 256;
  int64_t best = INT64_MAX;
  for (int i = 0; i < 4; ++i) {
    const int64_t per = (steps + (1 << i) - 1) >> i;
    if (most[i] <= 0 || per > gb300::fp4_linear_steps()) continue;
    const int64_t rounds = (tiles + most[i] - 1) / most[i], cost = rounds * per;
    if (cost < best) {
      best = cost;
      *c = Clusters{1 << i, int(tiles < most[i] ? tiles : most[i]), steps, per};
    }
  }
  return best != INT64_MAX;
}

// C = A B^T with the plan's partial sums at `partials` (after the counters at `ws`).
sgemm_status_t run_product(const Product& p, const fp4_matrix_t& A, const fp4_matrix_t& B, int dtype, void* C,
                           int64_t ldc, void* ws, void* partials, const LibDevice& d, cudaStream_t stream) {
  const gb300::Fp4TcTile t = gb300::fp4_tc_tile(p.shape);
  const fp4_matrix_t& R = t.swap ? B : A;
  const fp4_matrix_t& Q = t.swap ? A : B;
  const int64_t es = dtype_bytes(dtype);
  const int per_stage = int(64 / block_of(A.format));
  CUtensorMap maps[5];
  sgemm_status_t st = gb300::lib_encode_bytes(R.codes, R.rows, code_pitch(R.cols), R.ld, 128, &maps[0]);
  if (st == SGEMM_OK)
    st = gb300::lib_encode_bytes(Q.codes, Q.rows, code_pitch(Q.cols), Q.ld, t.cols / t.ctas, &maps[1]);
  for (int i = 0; i < 2 && st == SGEMM_OK; ++i) {
    const fp4_matrix_t& q = i ? Q : R;
    st = gb300::lib_encode_rows512(q.scales, scale_bytes(q.format, q.rows, q.cols) / 512, per_stage, &maps[2 + i]);
  }
  gb300::Fp4TcArgs a{};
  a.rows = int32_t(R.rows);
  a.cols = int32_t(Q.rows);
  a.out = C;
  a.ld = ldc;
  a.factor_r = R.factor;
  a.factor_c = Q.factor;
  a.partials = static_cast<float*>(partials);
  a.counters = static_cast<int32_t*>(ws);
  a.status = d.status;
  a.wait_limit_ns = d.wait_limit_ns;
  a.tma_out = !t.swap && stores_by_tma(C, ldc, Q.rows, es);
  a.tma_edge = Q.rows * es % 16 == 0;
  if (st == SGEMM_OK) {
    if (a.tma_out)
      st = gb300::lib_encode_bytes(C, A.rows, Q.rows * es, ldc * es, 32, &maps[4]);
    else
      maps[4] = maps[0];  // not used
  }
  if (st != SGEMM_OK) return st;
  return status_of(gb300::launch_fp4_tc(dtype, A.format, p.shape, maps, a, p.sc, p.grid, stream));
}

// C = 0 for an empty sum.
sgemm_status_t zero_output(int dtype, void* C, int64_t rows, int64_t cols, int64_t ldc, cudaStream_t stream) {
  const size_t es = size_t(dtype_bytes(dtype));
  return status_of(cudaMemset2DAsync(C, size_t(ldc) * es, 0, size_t(cols) * es, size_t(rows), stream));
}

}  // namespace

extern "C" {

sgemm_status_t fp4_layout(int format, int64_t rows, int64_t cols, int64_t* ld, int64_t* codes, int64_t* scales) try {
  sgemm_status_t st = check_format(format);
  if (st == SGEMM_OK) st = check_extent(rows, cols);
  if (st != SGEMM_OK) return st;
  if (ld) *ld = code_pitch(cols);
  if (codes) *codes = rows * code_pitch(cols);
  if (scales) *scales = scale_bytes(format, rows, cols);
  return SGEMM_OK;
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_quantize(int dtype, const void* x, int64_t ldx, const fp4_matrix_t* q, cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(q);
  if (st == SGEMM_OK) st = check_dense(dtype, x, q->rows, q->cols, ldx);
  if (st != SGEMM_OK) return st;
  const Range r = dense_range(dtype, x, q->rows, q->cols, ldx);
  for (const Range& out : {code_range(q), scale_range(q)})
    if (overlap(out, r) || overlap(out, factor_range(q->factor))) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || q->rows == 0 || q->cols == 0) return st;
  return status_of(gb300::launch_fp4_quantize(dtype, x, ldx, *q, d.sms, stream));
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_pack(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales,
                        const fp4_matrix_t* q, cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(q);
  if (st != SGEMM_OK) return st;
  LibDevice d;
  const int64_t blocks = (q->cols + block_of(q->format) - 1) / block_of(q->format);
  if (q->rows != 0 && q->cols != 0) {
    if (codes == nullptr || scales == nullptr || ld_codes < (q->cols + 1) / 2 || ld_scales < blocks)
      return SGEMM_ERR_INVALID_VALUE;
    const Range a = range(codes, (q->rows - 1) * ld_codes + (q->cols + 1) / 2);
    const Range b = range(scales, (q->rows - 1) * ld_scales + blocks);
    for (const Range& r : {code_range(q), scale_range(q)})
      if (overlap(a, r) || overlap(b, r)) return SGEMM_ERR_INVALID_VALUE;
  }
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || q->rows == 0 || q->cols == 0) return st;
  return status_of(gb300::launch_fp4_pack(codes, ld_codes, scales, ld_scales, *q, d.sms, stream));
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_dequantize(const fp4_matrix_t* q, int dtype, void* y, int64_t ldy, cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(q);
  if (st == SGEMM_OK) st = check_dense(dtype, y, q->rows, q->cols, ldy);
  if (st != SGEMM_OK) return st;
  const Range r = dense_range(dtype, y, q->rows, q->cols, ldy);
  if (overlap(r, q)) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || q->rows == 0 || q->cols == 0) return st;
  return status_of(gb300::launch_fp4_dequantize(*q, dtype, y, ldy, d.sms, stream));
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_gemm(const fp4_matrix_t* A, const fp4_matrix_t* B, int dtype, void* C, int64_t ldc,
                        cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(A);
  if (st == SGEMM_OK) st = check_quantized(B);
  if (st != SGEMM_OK) return st;
  if (A->format != B->format || A->cols != B->cols) return SGEMM_ERR_INVALID_VALUE;
  st = check_dense(dtype, C, A->rows, B->rows, ldc);
  if (st != SGEMM_OK) return st;
  const Range r = dense_range(dtype, C, A->rows, B->rows, ldc);
  if (overlap(r, A) || overlap(r, B)) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || A->rows == 0 || B->rows == 0) return st;
  if (A->cols == 0) return zero_output(dtype, C, A->rows, B->rows, ldc, stream);
  Product p;
  const int pairs = tc_pairs(d.dev);
  if (pairs < 0) return SGEMM_ERR_LAUNCH;
  if (!plan_product(A->rows, B->rows, A->cols, d.sms, pairs, dtype_bytes(dtype), C, ldc, &p)) return SGEMM_ERR_UNSUPPORTED;
  void* ws = nullptr;
  if (p.partial_bytes > 0) st = gb300::lib_workspace(d.dev, stream, gb300::kWorkspaceCounterBytes + p.partial_bytes, &ws);
  if (st != SGEMM_OK) return st;
  void* partials = ws ? static_cast<uint8_t*>(ws) + gb300::kWorkspaceCounterBytes : nullptr;
  return run_product(p, *A, *B, dtype, C, ldc, ws, partials, d, stream);
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_linear(int dtype, const void* x, int64_t ldx, int64_t M, const float* x_factor,
                          const fp4_matrix_t* W, void* y, int64_t ldy, cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(W);
  if (st == SGEMM_OK) st = check_dense(dtype, x, M, W->cols, ldx);
  if (st == SGEMM_OK) st = check_dense(dtype, y, M, W->rows, ldy);
  if (st != SGEMM_OK) return st;
  if (!aligned(x_factor, 4)) return SGEMM_ERR_INVALID_VALUE;
  const Range r = dense_range(dtype, y, M, W->rows, ldy);
  if (overlap(r, W) || overlap(r, factor_range(x_factor)) || overlap(r, dense_range(dtype, x, M, W->cols, ldx)))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || M == 0 || W->rows == 0) return st;
  fp4_matrix_t q{};
  q.format = W->format;
  q.rows = M;
  q.cols = W->cols;
  q.ld = code_pitch(W->cols);
  q.factor = x_factor;
  if (W->cols == 0) return zero_output(dtype, y, M, W->rows, ldy, stream);
  Clusters c;
  if (plan_linear(M, W->rows, W->cols, d.dev, &c)) {
    CUtensorMap map;
    st = gb300::lib_encode_bytes(W->codes, W->rows, code_pitch(W->cols), W->ld, 128, &map);
    if (st != SGEMM_OK) return st;
    gb300::Fp4LinearArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.x_factor = x_factor;
    a.scales = W->scales;
    a.w_factor = W->factor;
    a.y = y;
    a.ldy = ldy;
    a.tokens = int32_t(M);
    a.n = int32_t(W->rows);
    a.k = int32_t(W->cols);
    a.steps = int32_t(c.steps);
    a.ctas = c.ctas;
    a.per = int32_t(c.per);
    a.status = d.status;
    a.wait_limit_ns = d.wait_limit_ns;
    return status_of(gb300::launch_fp4_linear(dtype, W->format, map, a, c.clusters, stream));
  }
  Product p;
  const int pairs = tc_pairs(d.dev);
  if (pairs < 0) return SGEMM_ERR_LAUNCH;
  if (!plan_product(M, W->rows, W->cols, d.sms, pairs, dtype_bytes(dtype), y, ldy, &p)) return SGEMM_ERR_UNSUPPORTED;
  // Scratch: counters, partial sums, the codes and scales of x.
  const size_t code_at = gb300::kWorkspaceCounterBytes + (p.partial_bytes + 255) / 256 * 256;
  const size_t scale_at = code_at + size_t(M * q.ld + 255) / 256 * 256;
  void* ws = nullptr;
  st = gb300::lib_workspace(d.dev, stream, scale_at + size_t(scale_bytes(W->format, M, W->cols)), &ws);
  if (st != SGEMM_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  q.codes = base + code_at;
  q.scales = base + scale_at;
  if (gb300::launch_fp4_quantize(dtype, x, ldx, q, d.sms, stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
  return run_product(p, q, *W, dtype, y, ldy, ws, base + gb300::kWorkspaceCounterBytes, d, stream);
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_experts_layout(int format, int64_t experts, int64_t d, int64_t f, int64_t* gate_up_bytes,
                                  int64_t* down_bytes) try {
  sgemm_status_t st = check_format(format);
  if (st == SGEMM_OK) st = check_extent(d, f);
  if (st == SGEMM_OK) st = check_extent(experts, 0);
  if (st != SGEMM_OK) return st;
  if (experts > 1024) return SGEMM_ERR_UNSUPPORTED;
  if (gate_up_bytes) *gate_up_bytes = gb300::fp4_gate_up_bytes(format, experts, d, f);
  if (down_bytes) *down_bytes = gb300::fp4_down_bytes(format, experts, d, f);
  return SGEMM_OK;
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

static sgemm_status_t check_experts(const fp4_experts_t* w) {
  if (w == nullptr) return SGEMM_ERR_INVALID_VALUE;
  int64_t up = 0, down = 0;
  const sgemm_status_t st = fp4_experts_layout(w->format, w->experts, w->d, w->f, &up, &down);
  if (st != SGEMM_OK) return st;
  if ((up > 0 && (w->gate_up == nullptr || w->down == nullptr)) || !aligned(w->gate_up, 16) ||
      !aligned(w->down, 16) || !aligned(w->gate_up_factor, 4) || !aligned(w->down_factor, 4))
    return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

sgemm_status_t fp4_experts_pack(const fp4_matrix_t* gate_up, const fp4_matrix_t* down, const fp4_experts_t* w,
                                cudaStream_t stream) try {
  sgemm_status_t st = check_quantized(gate_up);
  if (st == SGEMM_OK) st = check_quantized(down);
  if (st == SGEMM_OK) st = check_experts(w);
  if (st != SGEMM_OK) return st;
  if (gate_up->format != w->format || down->format != w->format || gate_up->cols != w->d || down->cols != w->f ||
      gate_up->rows != w->experts * 2 * w->f || down->rows != w->experts * w->d)
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || w->experts == 0 || w->d == 0 || w->f == 0) return st;
  return status_of(gb300::launch_fp4_experts_pack(*gate_up, *down, *w, stream));
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

sgemm_status_t fp4_moe(int dtype, const void* x, int64_t ldx, int64_t M, const float* router, int64_t ldr,
                       const fp4_experts_t* w, int32_t top, int32_t renormalize, void* y, int64_t ldy, int32_t* ids,
                       float* p, cudaStream_t stream) try {
  sgemm_status_t st = check_experts(w);
  if (st == SGEMM_OK) st = check_dense(dtype, x, M, w->d, ldx);
  if (st == SGEMM_OK) st = check_dense(FP4_F32, router, w->experts, w->d, ldr);
  if (st == SGEMM_OK) st = check_dense(dtype, y, M, w->d, ldy);
  if (st != SGEMM_OK) return st;
  if (top < 1 || top > 32 || top > w->experts || !aligned(ids, 4) || !aligned(p, 4)) return SGEMM_ERR_INVALID_VALUE;
  if (w->d == 0 || w->f == 0) return SGEMM_ERR_INVALID_VALUE;
  int64_t up_bytes = 0, down_bytes = 0;
  fp4_experts_layout(w->format, w->experts, w->d, w->f, &up_bytes, &down_bytes);
  const Range outs[3] = {dense_range(dtype, y, M, w->d, ldy), range(ids, ids ? M * top * 4 : 0), range(p, p ? M * top * 4 : 0)};
  const Range ins[6] = {dense_range(dtype, x, M, w->d, ldx), dense_range(FP4_F32, router, w->experts, w->d, ldr),
                        range(w->gate_up, up_bytes),         range(w->down, down_bytes),
                        factor_range(w->gate_up_factor),     factor_range(w->down_factor)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& in : ins)
      if (overlap(outs[i], in)) return SGEMM_ERR_INVALID_VALUE;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return SGEMM_ERR_INVALID_VALUE;
  }
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || M == 0) return st;
  if (!moe_ready(d.dev)) return SGEMM_ERR_LAUNCH;
  const int64_t most = M < gb300::kMoeTokens ? M : gb300::kMoeTokens;
  const int64_t used = w->experts < most * top ? w->experts : most * top;
  // Stage counts of a phase are 32-bit numbers.
  if (used * ((w->f + 63) / 64) * ((w->d + 255) / 256) > 0x7fffffffLL ||
      used * ((w->f + 255) / 256) * ((w->d + 127) / 128) > 0x7fffffffLL)
    return SGEMM_ERR_UNSUPPORTED;
  const gb300::MoeScratch s = gb300::fp4_moe_scratch(dtype, w->format, most, w->experts, w->d, w->f, top, d.sms);
  void* ws = nullptr;
  st = gb300::lib_workspace(d.dev, stream, gb300::kWorkspaceCounterBytes + s.bytes, &ws);
  if (st != SGEMM_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws) + gb300::kWorkspaceCounterBytes;
  gb300::MoeArgs a{};
  a.ldx = ldx;
  a.router = router;
  a.ldr = ldr;
  a.gate_up = w->gate_up;
  a.down = w->down;
  a.gate_up_factor = w->format == FP4_NVFP4 ? w->gate_up_factor : nullptr;
  a.down_factor = w->format == FP4_NVFP4 ? w->down_factor : nullptr;
  a.ldy = ldy;
  a.experts = int32_t(w->experts);
  a.d = int32_t(w->d);
  a.f = int32_t(w->f);
  a.top = top;
  a.renormalize = renormalize;
  a.logits = reinterpret_cast<float*>(base + s.logits);
  a.x_exp = reinterpret_cast<int32_t*>(base + s.x_exp);
  a.x_norm = reinterpret_cast<float*>(base + s.x_norm);
  a.h_max = reinterpret_cast<uint32_t*>(base + s.h_max);
  a.h = reinterpret_cast<float*>(base + s.h);
  a.x_image = base + s.x_image;
  a.h_image = base + s.h_image;
  a.share = reinterpret_cast<uint64_t*>(base + s.share);
  a.bound = gb300::fp4_expert_bounds(*w);
  a.cols = s.cols;
  a.counters = static_cast<int32_t*>(ws);
  a.status = d.status;
  a.wait_limit_ns = d.wait_limit_ns;
  const int64_t bytes = dtype_bytes(dtype);
  for (int64_t t = 0; t < M; t += gb300::kMoeTokens) {
    a.tokens = int32_t(M - t < gb300::kMoeTokens ? M - t : gb300::kMoeTokens);
    a.x = static_cast<const uint8_t*>(x) + t * ldx * bytes;
    a.y = static_cast<uint8_t*>(y) + t * ldy * bytes;
    a.ids = ids ? ids + t * top : nullptr;
    a.p = p ? p + t * top : nullptr;
    if (gb300::launch_fp4_moe(dtype, w->format, a, d.sms, stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
  }
  return SGEMM_OK;
} catch (...) {  // no exception leaves a C entry: only the caches allocate
  return SGEMM_ERR_ALLOC;
}

}  // extern "C"
