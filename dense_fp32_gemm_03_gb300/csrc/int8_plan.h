// int8_plan.h -- which kernel computes a product of the 8-bit integer operators, and how the tiled one's work is cut.  Host
// code without calls of the CUDA runtime.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "int8_internal.h"

namespace gb300 {

constexpr int64_t int8_divide_up(int64_t n, int64_t d) { return (n + d - 1) / d; }

// A form of the tiled kernel: columns of a tile (of 256 rows); shares of k that a cluster's pairs can join among themselves;
// stages of k after which sums leave the accumulator (0: they stay for all of a share); whether it takes more than one term.
struct Int8TcForm {
  int cols, shares, run;
  bool terms;
};
constexpr Int8TcForm int8_tc_form(int shape) {
  return shape == kInt8Whole32    ? Int8TcForm{32, 4, 8, false}  // (of integers: 1024 products are exact)
         : shape == kInt8Whole64  ? Int8TcForm{64, 4, 8, false}
         : shape == kInt8Whole128 ? Int8TcForm{128, 4, 8, false}
         : shape == kInt8Bf16N128 || shape == kInt8F16N128       ? Int8TcForm{128, 4, 0, false}
         : shape == kInt8Bf16N256 || shape == kInt8F16N256       ? Int8TcForm{256, 1, 0, false}
         : shape == kInt8Bf16Runs256 || shape == kInt8F16Runs256 ? Int8TcForm{256, 1, 16, false}
                                                                 : Int8TcForm{128, 4, 4, true};
}

// The fewest clusters of each size that any form of the kernel can have at once: none if one form cannot have them.
class Int8LeastClusters {
 public:
  void take(int pairs, int clusters) {  // of 1, 2 or 4 pairs
    int& least = least_[pairs / 2];
    if (least < 0 || clusters < least) least = clusters;
  }
  Int8TcClusters clusters() const { return {std::max(least_[0], 0), std::max(least_[1], 0), std::max(least_[2], 0)}; }

 private:
  int least_[3] = {-1, -1, -1};  // (not known yet)
};

// Tokens whose sums may stay in one accumulator of the tensor core.  An MMA adds 16 of them and cuts off what is below the
// accumulator's last place: with sums of one sign 6.5e-9 of the sum a token were measured to be lost (over 262144 tokens 1.7e-3).
// For results of 32 bits sums leave it every 512 tokens.  For those of 16 bits the loss stays below 1/30 of half a step of the
// type (2^-8 for bfloat16, 2^-11 for 16-bit floats), 16384 and 2048 tokens; beyond, sums leave it as well, in tiles of 128 columns or every
// 2048 tokens in tiles of 256 (16384 x 4096 x 4096 fp16 343 us, with all in one accumulator 323).
constexpr int64_t int8_most_tokens(int dtype) { return dtype == INT8_F32 ? 512 : dtype == INT8_BF16 ? 16384 : 2048; }

// The tiles, and the shares that k is cut into where there are fewer tiles than pairs of CTAs, that are estimated to
// be fastest (us, fitted to 41 products timed with every choice: the chosen ones are within 4 % of the best, and within 5 %
// in 31 others).  A stage of 128 of k takes its MMAs, 0.53 for 256 columns and 0.28 for 128 or fewer (reading `a` from tensor
// memory takes as long), and at least what turning `a` to 16 bits takes, 0.37 with a checkpoint's units; a tile fills and
// empties the pipeline (1.5), and the last one is stored.  Shares meet within a cluster, or are written and added by a kernel
// of its own, 4 bytes each way: 14.2 and 16.6 us for 4096 x 1024 x 1024 bf16, one share 18.4.  Equal ones: the narrower
// tiles, which read less of b.  A form whose sums stay in the accumulator takes at most `most_steps` stages a share.
// False if there is no way.
inline bool int8_plan_tiles(std::initializer_list<Int8TcShape> shapes, int64_t rows, int64_t cols, int64_t depth, int terms, bool units,
                            int64_t most_steps, const Int8TcClusters& most, Int8TcArgs* a, Int8TcShape* best, double* estimate) {
  const int64_t steps = int8_divide_up(depth, kInt8TcStep), tr = int8_divide_up(rows, 256), pairs = most.pairs;
  if (pairs <= 0) return false;
  a->rows = int32_t(rows);
  a->cols = int32_t(cols);
  a->depth = int32_t(depth);
  a->steps = int32_t(steps);
  a->terms = terms;
  double least = 0.0;
  for (const Int8TcShape shape : shapes) {
    const Int8TcForm form = int8_tc_form(shape);
    const int64_t n = form.cols, tc = int8_divide_up(cols, n), tiles = tr * tc;
    if (tiles > 0x3fffffffLL || (terms > 1 && !form.terms)) continue;
    const int64_t needed = form.run ? 1 : int8_divide_up(steps, most_steps);
    const bool wide = form.run && n == 256;  // (reads its one accumulator between the MMAs of two runs, and stores from 32 bits)
    const double stage = std::max(units ? 0.37 : 0.0, double(terms) * std::max(0.28, double(n) * ((wide ? 0.56 : 0.53) / 256)));
    const double last = std::min(3.0, 0.02 * double(n - 32)) + (wide ? 3.0 : 0.0);
    auto consider = [&](int64_t splits, bool join) {
      if (splits < needed) return;
      const double us = double(int8_divide_up(tiles * splits, pairs)) * (double(int8_divide_up(steps, splits)) * stage + 1.5) + last +
                        (join ? 0.3 + 0.25 * double(splits) : splits > 1 ? 2.5 + double(splits) * double(rows) * double(cols) * 1e-6 : 0.0);
      if (least > 0.0 && us >= least) return;
      least = us;
      *best = shape;
      a->run = form.run;
      a->tiles_r = int32_t(tr);
      a->tiles_c = int32_t(tc);
      a->splits = int32_t(splits);
      a->units = int32_t(tiles * splits);
      a->join = join;
    };
    consider(1, false);
    for (int64_t splits = 2; splits <= form.shares; splits *= 2)
      if (tiles <= (splits == 2 ? most.twos : most.fours) && splits <= steps) consider(splits, true);
    if (std::min(pairs / tiles, steps / 4) > 1) consider(std::min(pairs / tiles, steps / 4), false);
  }
  *estimate = least;
  return least > 0.0;
}

// ---- products of integers: y = X W^T of M tokens, W N x K
// us, fitted to 60 products of 16 to 512 tokens: the launch, what a block of int8_few.cu loads and converts, what it adds up and
// stores.  (A kernel before it that quantises takes 2 more.)
inline double int8_few_estimate(int64_t tokens, int64_t n, int64_t k) {
  return 1.8 + double(tokens) * double(n) * (double(k) * 2.2e-8 + 5e-6);
}

// What computes it: int8_few.cu, or tiles as planned.
struct Int8Plan {
  bool ok, small;  // small: int8_few.cu or int8_grad.cu
  Int8TcShape shape;
  Int8TcArgs a;
};
// Up to eight tokens int8_few.cu.  More go there eight by eight where that is estimated to be faster: 300 x 520 x 200 3.4 us (in
// tiles 6.1), 512 x 1024 x 1024 13.5 (8.7).  4 us: the kernel that prepares b, and launches.
inline Int8Plan int8_plan_product(int64_t m, int64_t n, int64_t k, bool quantised, const Int8TcClusters& most) {
  Int8Plan p{true, true, kInt8Whole32, {}};
  if (m <= kInt8FewTokens) return p;
  double estimate = 0.0;
  p.ok = int8_plan_tiles({kInt8Whole32, kInt8Whole64, kInt8Whole128}, n, m, k, 1, false, 0, most, &p.a, &p.shape, &estimate);
  p.small = p.ok && int8_few_estimate(m, n, k) + (quantised ? 0.0 : 2.0) < estimate + 4.0;
  return p;
}

// ---- weight gradients: dW (n x cols) of `tokens` tokens kept as `kept`, of type `dtype`
constexpr int int8_terms(int dtype) { return dtype == INT8_F32 ? 3 : 1; }  // of 16 bits that hold a value of dY

// us of int8_grad.cu, fitted to 15 sizes of each form: the launch, a warp's steps one after the other, a block, and a block's
// steps.  vec: dY's rows are read 16 bytes at a time.
inline double int8_grad_estimate(int kept, bool vec, int64_t tokens, int64_t n, int64_t cols) {
  const int64_t steps = int8_divide_up(tokens, kInt8GradStep);
  const double rounds = double(int8_divide_up(steps, kInt8GradWarps));
  const double blocks = double(int8_divide_up(cols, kInt8GradTile) * int8_divide_up(n, kInt8GradTile));
  if (kept == INT8_F32) return 2.0 + 2.5 * rounds + blocks * double(steps) * 0.0035;
  return vec ? 1.5 + 0.9 * rounds + blocks * (0.0027 + 0.00047 * double(steps))
             : 1.4 + 1.4 * rounds + blocks * (0.003 + 0.0005 * double(steps));
}

// in_place: the tiled kernel reads dY where it is.  int8_grad.cu where that takes so little that launches are most of it (2.2 us, with
// a kernel before it 3), and its warps' accumulators do not take too many tokens.
inline Int8Plan int8_plan_gradient(int kept, int dtype, bool in_place, bool vec, int64_t tokens, int64_t n, int64_t cols,
                                   const Int8TcClusters& most) {
  Int8Plan p{true, false, kInt8Bf16Runs, {}};
  const bool half = kept == INT8_F16;
  const int64_t most_tokens = int8_most_tokens(dtype);
  double estimate = 0.0;
  auto tiles = [&](std::initializer_list<Int8TcShape> shapes) {
    p.ok = int8_plan_tiles(shapes, cols, n, tokens, int8_terms(kept), true, most_tokens / kInt8TcStep, most, &p.a, &p.shape, &estimate);
  };
  if (dtype == INT8_F32)
    tiles({half ? kInt8F16Runs : kInt8Bf16Runs});
  else if (half)
    tiles({kInt8F16N128, kInt8F16Runs, kInt8F16N256, kInt8F16Runs256});
  else
    tiles({kInt8Bf16N128, kInt8Bf16Runs, kInt8Bf16N256, kInt8Bf16Runs256});
  p.small = p.ok && tokens <= kInt8GradWarps * most_tokens &&
            int8_grad_estimate(kept, vec, tokens, n, cols) < estimate + (in_place ? 2.2 : 3.0);
  return p;
}

}  // namespace gb300
