// int8_api.cu -- host side of the 8-bit integer operators' C ABI
// (include/int8.h): argument validation, scratch and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <map>
#include <mutex>

#include "int8.h"
#include "int8_internal.h"
#include "int8_plan.h"
#include "sgemm_internal.h"

namespace {

using gb300::LibDevice;

// Rows and columns: element counts of a row stay within 32 bits.
constexpr int64_t kMaxExtent = int64_t(1) << 30;
constexpr int64_t kMaxDepth = 131071;  // 128 * 128 * 131071 < 2^31

int64_t dtype_bytes(int dtype) { return dtype == INT8_F32 ? 4 : 2; }
int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
sgemm_status_t status_of(cudaError_t e) { return e == cudaSuccess ? SGEMM_OK : SGEMM_ERR_LAUNCH; }

sgemm_status_t check_extent(int64_t a, int64_t b) {
  if (a < 0 || b < 0) return SGEMM_ERR_INVALID_VALUE;
  return a > kMaxExtent || b > kMaxExtent ? SGEMM_ERR_UNSUPPORTED : SGEMM_OK;
}

bool known(int dtype) { return dtype >= INT8_F32 && dtype <= INT8_F16; }

// An unquantised rows x cols matrix.
sgemm_status_t check_dense(int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  if (!known(dtype)) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(rows, cols);
  if (st != SGEMM_OK || rows == 0 || cols == 0) return st;
  if (p == nullptr || ld < cols || !aligned(p, size_t(dtype_bytes(dtype)))) return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

sgemm_status_t check_rows(const int8_matrix_t* q) {
  if (q == nullptr) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(q->rows, q->cols);
  if (st != SGEMM_OK || q->rows == 0) return st;
  if (q->scales == nullptr || !aligned(q->scales, 4)) return SGEMM_ERR_INVALID_VALUE;
  if (q->cols == 0) return SGEMM_OK;
  if (q->codes == nullptr || !aligned(q->codes, 16) || q->ld < round_up(q->cols, 16) || q->ld % 16 != 0)
    return SGEMM_ERR_INVALID_VALUE;
  return SGEMM_OK;
}

// Rows of a checkpoint's arrays, and entries of one.
struct Lines {
  int64_t codes, code_entries, units, unit_entries;
};
Lines lines_of(int order, int64_t rows, int64_t cols) {
  const int64_t blocks = (cols + 31) / 32;
  return order == INT8_CHANNELS ? Lines{cols, rows, blocks, rows} : Lines{rows, cols, rows, blocks};
}

sgemm_status_t check_kept(const int8_checkpoint_t* c, int order) {
  if (c == nullptr || !known(c->dtype) || (c->order != INT8_CHANNELS && c->order != INT8_TOKENS)) return SGEMM_ERR_INVALID_VALUE;
  if (order >= 0 && c->order != order) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(c->rows, c->cols);
  if (st != SGEMM_OK || c->rows == 0 || c->cols == 0) return st;
  const Lines n = lines_of(c->order, c->rows, c->cols);
  if (c->codes == nullptr || c->units == nullptr || !aligned(c->codes, 16) || !aligned(c->units, 16) ||
      c->ld < round_up(n.code_entries, 16) || c->ld % 16 != 0 || c->ld_units < round_up(n.unit_entries, 8) ||
      c->ld_units % 8 != 0)
    return SGEMM_ERR_INVALID_VALUE;
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
Range code_range(const int8_matrix_t* q) { return range(q->codes, q->rows && q->cols ? (q->rows - 1) * q->ld + round_up(q->cols, 16) : 0); }
Range scale_range(const int8_matrix_t* q) { return range(q->scales, q->rows * 4); }
Range code_range(const int8_checkpoint_t* c) {
  const Lines n = lines_of(c->order, c->rows, c->cols);
  return range(c->codes, c->rows && c->cols ? (n.codes - 1) * c->ld + round_up(n.code_entries, 16) : 0);
}
Range unit_range(const int8_checkpoint_t* c) {
  const Lines n = lines_of(c->order, c->rows, c->cols);
  return range(c->units, c->rows && c->cols ? 2 * ((n.units - 1) * c->ld_units + round_up(n.unit_entries, 8)) : 0);
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool overlap_any(Range a, std::initializer_list<Range> others) {
  for (const Range& b : others)
    if (overlap(a, b)) return true;
  return false;
}
// Whether the rows of two matrices (of bytes_a and bytes_b each) share memory; rows of one may lie between the other's (parts of
// the rows of one tensor).
bool rows_overlap(int64_t rows, int64_t bytes_a, const void* a, int64_t lda, int64_t bytes_b, const void* b, int64_t ldb) {
  const Range ra = range(a, (rows - 1) * lda + bytes_a), rb = range(b, (rows - 1) * ldb + bytes_b);
  if (rows <= 0 || bytes_a <= 0 || bytes_b <= 0 || !overlap(ra, rb)) return false;
  if (lda != ldb) return true;
  const int64_t shift = (int64_t(rb.lo - ra.lo) % lda + lda) % lda;  // from a row of a to the next of b's
  return shift < bytes_a || shift + bytes_b > lda;
}
bool rows_overlap(int64_t rows, int64_t bytes, const void* a, int64_t lda, const void* b, int64_t ldb) {
  return rows_overlap(rows, bytes, a, lda, bytes, b, ldb);
}

// C = 0 for an empty sum.
sgemm_status_t zero_output(int dtype, void* C, int64_t rows, int64_t cols, int64_t ldc, cudaStream_t stream) {
  const size_t es = size_t(dtype_bytes(dtype));
  return status_of(cudaMemset2DAsync(C, size_t(ldc) * es, 0, size_t(cols) * es, size_t(rows), stream));
}

// Places in the workspace, after the counters.
struct Scratch {
  size_t bytes = gb300::kWorkspaceCounterBytes;
  size_t take(int64_t n) {
    const size_t at = bytes;
    bytes += size_t(round_up(n, 256));
    return at;
  }
};

// ------------------------------------------------------------------- products
std::mutex g_mu;
std::map<int, gb300::Int8TcClusters> g_clusters;  // by device; no pairs: not to be had

gb300::Int8TcClusters tc_clusters(int dev) {
  std::lock_guard<std::mutex> lock(g_mu);
  auto it = g_clusters.find(dev);
  if (it == g_clusters.end()) {
    gb300::Int8TcClusters n;
    if (!gb300::int8_tc_prepare(&n)) n = gb300::Int8TcClusters{};
    it = g_clusters.emplace(dev, n).first;
  }
  return it->second;
}

// A product's operands (int8_internal.h), before it is planned.
struct Operands {
  const int8_t* a;
  int64_t lda;
  const uint16_t* units;  // NULL: integers
  int64_t ldu;
  const uint16_t* b;
  int64_t ldb;
  int terms;
};

sgemm_status_t no_plan(const gb300::Int8TcClusters& most) { return most.pairs > 0 ? SGEMM_ERR_UNSUPPORTED : SGEMM_ERR_LAUNCH; }
size_t partial_bytes(const gb300::Int8TcArgs& a) {
  return a.splits > 1 && !a.join ? size_t(a.splits) * size_t(a.rows) * size_t(a.cols) * 4 : 0;
}

sgemm_status_t run_product(gb300::Int8TcShape shape, const Operands& o, gb300::Int8TcArgs a, int pairs, const LibDevice& d,
                           cudaStream_t stream) {
  CUtensorMap maps[3];
  const int64_t cols8 = round_up(a.cols, 8), depth8 = round_up(a.depth, 8);
  sgemm_status_t st = gb300::lib_encode_bytes(o.a, a.rows, round_up(a.depth, 16), o.lda, 128, &maps[0]);
  if (st != SGEMM_OK) return st;
  if (o.units) {
    st = gb300::lib_encode_bytes(o.units, (a.rows + 31) / 32, 2 * depth8, 2 * o.ldu, 4, &maps[1]);
    if (st == SGEMM_OK) st = gb300::lib_encode_bytes(o.b, int64_t(o.terms) * a.depth, 2 * cols8, 2 * o.ldb, int(gb300::kInt8TcStep), &maps[2]);
  } else {
    maps[1] = maps[0];  // not used
    st = gb300::lib_encode_bytes(o.b, a.cols, 2 * depth8, 2 * o.ldb, gb300::int8_tc_form(shape).cols / 2, &maps[2]);
  }
  if (st != SGEMM_OK) return st;
  a.status = d.status;
  a.wait_limit_ns = d.wait_limit_ns;
  return status_of(gb300::launch_int8_tc(shape, maps, a, pairs, stream));
}

// C (M x N, row stride ldc) = A B^T, from A's rows as 16-bit floats or, with x, quantised on the way.
sgemm_status_t integer_product(const int8_matrix_t* A, int dtype_x, const void* x, int64_t ldx, int64_t M, const int8_matrix_t& B,
                               int dtype, void* C, int64_t ldc, const LibDevice& d, cudaStream_t stream) {
  const gb300::Int8TcClusters most = M <= gb300::kInt8FewTokens ? gb300::Int8TcClusters{} : tc_clusters(d.dev);
  const gb300::Int8Plan p = gb300::int8_plan_product(M, B.rows, B.cols, A != nullptr, most);
  if (!p.ok) return no_plan(most);
  if (p.small) {
    gb300::Int8FewArgs f{};
    f.w = B.codes;
    f.ldw = B.ld;
    f.scale_w = B.scales;
    f.y = C;
    f.ldy = ldc;
    f.n = int32_t(B.rows);
    f.k = int32_t(B.cols);
    f.tokens = int32_t(M);
    f.dtype = dtype;
    if (A) {
      f.x = A->codes;
      f.ldx = A->ld;
      f.scale_x = A->scales;
      return status_of(gb300::launch_int8_few(-1, f, d.sms, stream));
    }
    if (gb300::int8_few_quantises(M, B.rows, B.cols, d.sms)) {
      f.x = x;
      f.vec = aligned(x, 16);
      return status_of(gb300::launch_int8_few(dtype_x, f, d.sms, stream));
    }
    Scratch s;
    const int64_t ld = round_up(B.cols, 16);
    const size_t scales_at = s.take(M * 4), tokens_at = s.take(M * ld);
    void* ws = nullptr;
    const sgemm_status_t st = gb300::lib_workspace(d.dev, stream, s.bytes, &ws);
    if (st != SGEMM_OK) return st;
    uint8_t* base = static_cast<uint8_t*>(ws);
    const int8_matrix_t tokens{M, B.cols, reinterpret_cast<int8_t*>(base + tokens_at), ld, reinterpret_cast<float*>(base + scales_at)};
    if (gb300::launch_int8_quantize(dtype_x, x, ldx, tokens, stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
    f.x = tokens.codes;
    f.ldx = ld;
    f.scale_x = tokens.scales;
    f.early = 1;
    return status_of(gb300::launch_int8_few(-1, f, d.sms, stream));
  }
  gb300::Int8TcArgs a = p.a;
  const int64_t ld16 = round_up(B.cols, 64);  // whole lines of 128 bytes (16384 x 1024 x 4104: 166 us in multiples of 8, 143)
  Scratch s;
  const size_t scales_at = s.take(M * 4), rows_at = s.take(M * ld16 * 2), partials_at = s.take(int64_t(partial_bytes(a)));
  void* ws = nullptr;
  const sgemm_status_t st = gb300::lib_workspace(d.dev, stream, s.bytes, &ws);
  if (st != SGEMM_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  uint16_t* rows16 = reinterpret_cast<uint16_t*>(base + rows_at);
  float* scales = reinterpret_cast<float*>(base + scales_at);
  const cudaError_t e = A ? gb300::launch_int8_widen(*A, rows16, ld16, d.sms, stream)
                          : gb300::launch_int8_rows16(dtype_x, x, ldx, M, B.cols, rows16, ld16, scales, stream);
  if (e != cudaSuccess) return SGEMM_ERR_LAUNCH;
  a.scale_r = B.scales;
  a.scale_c = A ? A->scales : scales;
  a.dtype = dtype;
  a.out = C;
  a.ld = ldc;
  a.early = 1;
  a.partials = reinterpret_cast<uint32_t*>(base + partials_at);
  return run_product(p.shape, Operands{B.codes, B.ld, nullptr, 0, rows16, ld16, 1}, a, most.pairs, d, stream);
}

}  // namespace

// No exception leaves a C entry: only the caches allocate.
#define GB300_INT8_CATCH \
  catch (...) { return SGEMM_ERR_ALLOC; }

extern "C" {

sgemm_status_t int8_quantize(int dtype, const void* x, int64_t ldx, const int8_matrix_t* q, cudaStream_t stream) try {
  sgemm_status_t st = check_rows(q);
  if (st == SGEMM_OK) st = check_dense(dtype, x, q->rows, q->cols, ldx);
  if (st != SGEMM_OK) return st;
  const Range in = dense_range(dtype, x, q->rows, q->cols, ldx);
  if (overlap_any(in, {code_range(q), scale_range(q)}) || overlap(code_range(q), scale_range(q))) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || q->rows == 0) return st;
  return status_of(gb300::launch_int8_quantize(dtype, x, ldx, *q, stream));
} GB300_INT8_CATCH

sgemm_status_t int8_dequantize(const int8_matrix_t* q, int dtype, void* y, int64_t ldy, cudaStream_t stream) try {
  sgemm_status_t st = check_rows(q);
  if (st == SGEMM_OK) st = check_dense(dtype, y, q->rows, q->cols, ldy);
  if (st != SGEMM_OK) return st;
  if (overlap_any(dense_range(dtype, y, q->rows, q->cols, ldy), {code_range(q), scale_range(q)})) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || q->rows == 0 || q->cols == 0) return st;
  return status_of(gb300::launch_int8_dequantize(*q, dtype, y, ldy, d.sms, stream));
} GB300_INT8_CATCH

sgemm_status_t int8_gemm(const int8_matrix_t* A, const int8_matrix_t* B, int dtype, void* C, int64_t ldc,
                         cudaStream_t stream) try {
  sgemm_status_t st = check_rows(A);
  if (st == SGEMM_OK) st = check_rows(B);
  if (st != SGEMM_OK) return st;
  if (A->cols != B->cols) return SGEMM_ERR_INVALID_VALUE;
  st = check_dense(dtype, C, A->rows, B->rows, ldc);
  if (st != SGEMM_OK) return st;
  if (A->cols > kMaxDepth) return SGEMM_ERR_UNSUPPORTED;
  if (overlap_any(dense_range(dtype, C, A->rows, B->rows, ldc), {code_range(A), scale_range(A), code_range(B), scale_range(B)}))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || A->rows == 0 || B->rows == 0) return st;
  if (A->cols == 0) return zero_output(dtype, C, A->rows, B->rows, ldc, stream);
  return integer_product(A, 0, nullptr, 0, A->rows, *B, dtype, C, ldc, d, stream);
} GB300_INT8_CATCH

sgemm_status_t int8_linear(int dtype, const void* x, int64_t ldx, int64_t M, const int8_matrix_t* W, void* y,
                           int64_t ldy, cudaStream_t stream) try {
  sgemm_status_t st = check_rows(W);
  if (st == SGEMM_OK) st = check_dense(dtype, x, M, W->cols, ldx);
  if (st == SGEMM_OK) st = check_dense(dtype, y, M, W->rows, ldy);
  if (st != SGEMM_OK) return st;
  if (W->cols > kMaxDepth) return SGEMM_ERR_UNSUPPORTED;
  const int64_t es = dtype_bytes(dtype);
  if (overlap_any(dense_range(dtype, y, M, W->rows, ldy), {code_range(W), scale_range(W)}) ||
      rows_overlap(M, W->rows * es, y, ldy * es, W->cols * es, x, ldx * es))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || M == 0 || W->rows == 0) return st;
  if (W->cols == 0) return zero_output(dtype, y, M, W->rows, ldy, stream);
  return integer_product(nullptr, dtype, x, ldx, M, *W, dtype, y, ldy, d, stream);
} GB300_INT8_CATCH

sgemm_status_t int8_checkpoint_layout(int order, int64_t rows, int64_t cols, int64_t* ld, int64_t* ld_units,
                                      int64_t* code_bytes, int64_t* unit_bytes) try {
  if (order != INT8_CHANNELS && order != INT8_TOKENS) return SGEMM_ERR_INVALID_VALUE;
  const sgemm_status_t st = check_extent(rows, cols);
  if (st != SGEMM_OK) return st;
  const Lines n = lines_of(order, rows, cols);
  const int64_t pitch = round_up(n.code_entries, 16), units = round_up(n.unit_entries, 8);
  if (ld) *ld = pitch;
  if (ld_units) *ld_units = units;
  if (code_bytes) *code_bytes = n.codes * pitch;
  if (unit_bytes) *unit_bytes = n.units * units * 2;
  return SGEMM_OK;
} GB300_INT8_CATCH

sgemm_status_t int8_checkpoint(const void* x, int64_t ldx, const int8_checkpoint_t* c, cudaStream_t stream) try {
  sgemm_status_t st = check_kept(c, INT8_CHANNELS);
  if (st == SGEMM_OK) st = check_dense(c->dtype, x, c->rows, c->cols, ldx);
  if (st != SGEMM_OK) return st;
  if (overlap_any(dense_range(c->dtype, x, c->rows, c->cols, ldx), {code_range(c), unit_range(c)}) ||
      overlap(code_range(c), unit_range(c)))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || c->rows == 0 || c->cols == 0) return st;
  return status_of(gb300::launch_int8_keep(x, ldx, *c, stream));
} GB300_INT8_CATCH

sgemm_status_t int8_restore(const int8_checkpoint_t* c, int dtype, void* y, int64_t ldy, cudaStream_t stream) try {
  sgemm_status_t st = check_kept(c, -1);
  if (st == SGEMM_OK) st = check_dense(dtype, y, c->rows, c->cols, ldy);
  if (st != SGEMM_OK) return st;
  if (overlap_any(dense_range(dtype, y, c->rows, c->cols, ldy), {code_range(c), unit_range(c)})) return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || c->rows == 0 || c->cols == 0) return st;
  return status_of(gb300::launch_int8_restore(*c, dtype, y, ldy, d.sms, stream));
} GB300_INT8_CATCH

sgemm_status_t int8_weight_grad(const void* dy, int64_t lddy, int64_t N, const int8_checkpoint_t* c, int dtype,
                                int32_t accumulate, void* dw, int64_t ldw, cudaStream_t stream) try {
  sgemm_status_t st = check_kept(c, INT8_CHANNELS);
  if (st == SGEMM_OK) st = check_dense(c->dtype, dy, c->rows, N, lddy);
  if (st == SGEMM_OK) st = check_dense(dtype, dw, N, c->cols, ldw);
  if (st != SGEMM_OK) return st;
  if (dtype != c->dtype && dtype != INT8_F32) return SGEMM_ERR_INVALID_VALUE;
  // A row's bytes stay within 31 bits, and a tile's tokens within a quarter of the kernel's time limit for a wait.
  if (c->rows > kMaxExtent / 8 || N > kMaxExtent / 2) return SGEMM_ERR_UNSUPPORTED;
  if (overlap_any(dense_range(dtype, dw, N, c->cols, ldw), {code_range(c), unit_range(c), dense_range(c->dtype, dy, c->rows, N, lddy)}))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || N == 0 || c->cols == 0) return st;
  if (c->rows == 0) return accumulate ? SGEMM_OK : zero_output(dtype, dw, N, c->cols, ldw, stream);
  const gb300::Int8TcClusters most = tc_clusters(d.dev);
  const int terms = gb300::int8_terms(c->dtype);
  const bool in_place = terms == 1 && aligned(dy, 16) && (lddy % 8 == 0 || c->rows == 1);
  const gb300::Int8GradArgs g{c->codes, c->ld, c->units, c->ld_units, dy, lddy, int32_t(c->rows), int32_t(c->cols), int32_t(N),
                              dtype, accumulate != 0, dw, ldw};
  const gb300::Int8Plan p = gb300::int8_plan_gradient(c->dtype, dtype, in_place, gb300::int8_grad_vec(g), c->rows, N, c->cols, most);
  if (!p.ok) return no_plan(most);
  if (p.small) return status_of(gb300::launch_int8_grad(c->dtype, g, stream));
  gb300::Int8TcArgs a = p.a;
  Operands o{c->codes, c->ld, c->units, c->ld_units, static_cast<const uint16_t*>(dy), round_up(lddy, 8), terms};
  if (!in_place) o.ldb = round_up(N, 64);
  Scratch s;
  const size_t terms_at = s.take(in_place ? 0 : terms * c->rows * o.ldb * 2), partials_at = s.take(int64_t(partial_bytes(a)));
  void* ws = nullptr;
  st = gb300::lib_workspace(d.dev, stream, s.bytes, &ws);
  if (st != SGEMM_OK) return st;
  uint8_t* base = static_cast<uint8_t*>(ws);
  if (!in_place) {
    uint16_t* terms_out = reinterpret_cast<uint16_t*>(base + terms_at);
    o.b = terms_out;
    if (gb300::launch_int8_split(c->dtype, dy, lddy, c->rows, N, terms_out, o.ldb, d.sms, stream) != cudaSuccess) return SGEMM_ERR_LAUNCH;
  }
  a.early = !in_place;
  a.dtype = dtype;
  a.accumulate = accumulate != 0;
  a.out = dw;
  a.ld = ldw;
  a.partials = reinterpret_cast<uint32_t*>(base + partials_at);
  return run_product(p.shape, o, a, most.pairs, d, stream);
} GB300_INT8_CATCH

sgemm_status_t int8_swiglu(int dtype, int64_t M, int64_t F, const void* gate, int64_t ld_gate, const void* up,
                           int64_t ld_up, void* h, int64_t ld_h, const int8_checkpoint_t* kept_gate,
                           const int8_checkpoint_t* kept_up, cudaStream_t stream) try {
  sgemm_status_t st = check_dense(dtype, gate, M, F, ld_gate);
  if (st == SGEMM_OK) st = check_dense(dtype, up, M, F, ld_up);
  if (st == SGEMM_OK) st = check_dense(dtype, h, M, F, ld_h);
  for (const int8_checkpoint_t* c : {kept_gate, kept_up}) {
    if (st == SGEMM_OK) st = check_kept(c, INT8_TOKENS);
    if (st == SGEMM_OK && (c->dtype != dtype || c->rows != M || c->cols != F)) st = SGEMM_ERR_INVALID_VALUE;
  }
  if (st != SGEMM_OK) return st;
  const Range g = dense_range(dtype, gate, M, F, ld_gate), u = dense_range(dtype, up, M, F, ld_up);
  const Range kg = code_range(kept_gate), ug = unit_range(kept_gate), ku = code_range(kept_up), uu = unit_range(kept_up);
  const int64_t es = dtype_bytes(dtype);
  if (overlap_any(kg, {g, u, ug, ku, uu}) || overlap_any(ug, {g, u, ku, uu}) || overlap_any(ku, {g, u, uu}) || overlap_any(uu, {g, u}) ||
      overlap_any(dense_range(dtype, h, M, F, ld_h), {kg, ug, ku, uu}) || rows_overlap(M, F * es, h, ld_h * es, gate, ld_gate * es) ||
      rows_overlap(M, F * es, h, ld_h * es, up, ld_up * es))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || M == 0 || F == 0) return st;
  return status_of(gb300::launch_int8_swiglu(dtype, M, F, gate, ld_gate, up, ld_up, h, ld_h, *kept_gate, *kept_up, d.sms, stream));
} GB300_INT8_CATCH

sgemm_status_t int8_swiglu_backward(const void* dh, int64_t ld_dh, const int8_checkpoint_t* kept_gate,
                                    const int8_checkpoint_t* kept_up, void* dgate, int64_t ld_dgate, void* dup,
                                    int64_t ld_dup, cudaStream_t stream) try {
  sgemm_status_t st = check_kept(kept_gate, INT8_TOKENS);
  if (st == SGEMM_OK) st = check_kept(kept_up, INT8_TOKENS);
  if (st != SGEMM_OK) return st;
  const int dtype = kept_gate->dtype;
  const int64_t M = kept_gate->rows, F = kept_gate->cols, es = dtype_bytes(dtype);
  if (kept_up->dtype != dtype || kept_up->rows != M || kept_up->cols != F) return SGEMM_ERR_INVALID_VALUE;
  st = check_dense(dtype, dh, M, F, ld_dh);
  if (st == SGEMM_OK) st = check_dense(dtype, dgate, M, F, ld_dgate);
  if (st == SGEMM_OK) st = check_dense(dtype, dup, M, F, ld_dup);
  if (st != SGEMM_OK) return st;
  for (const Range& out : {dense_range(dtype, dgate, M, F, ld_dgate), dense_range(dtype, dup, M, F, ld_dup)})
    if (overlap_any(out, {code_range(kept_gate), unit_range(kept_gate), code_range(kept_up), unit_range(kept_up)}))
      return SGEMM_ERR_INVALID_VALUE;
  if (rows_overlap(M, F * es, dgate, ld_dgate * es, dup, ld_dup * es) || rows_overlap(M, F * es, dgate, ld_dgate * es, dh, ld_dh * es) ||
      rows_overlap(M, F * es, dup, ld_dup * es, dh, ld_dh * es))
    return SGEMM_ERR_INVALID_VALUE;
  LibDevice d;
  st = gb300::lib_device(&d);
  if (st != SGEMM_OK || M == 0 || F == 0) return st;
  return status_of(gb300::launch_int8_swiglu_backward(dh, ld_dh, *kept_gate, *kept_up, dgate, ld_dgate, dup, ld_dup, d.sms, stream));
} GB300_INT8_CATCH

}  // extern "C"
