// Host probe of which kernel computes a product of the 8-bit integer operators, for tests/int8_plans.py.
//
// Reads lines "kind kept dtype in_place vec m n k pairs twos fours" from stdin (kind 0: a product of m tokens, n channels and
// k columns, `kept` whether its tokens are integers already; 1: a weight gradient of m tokens, n columns of dY and k channels) and
// prints "ok small shape cols run splits join units run_taken tiles_r tiles_c" of the plan.  The functions are those that
// the library calls.
#include <cstdio>

#include "int8_plan.h"

int main() {
  int kind, kept, dtype, in_place, vec;
  long long m, n, k;
  gb300::Int8TcClusters most;
  while (std::scanf("%d %d %d %d %d %lld %lld %lld %d %d %d", &kind, &kept, &dtype, &in_place, &vec, &m, &n, &k, &most.pairs,
                    &most.twos, &most.fours) == 11) {
    const gb300::Int8Plan p = kind == 0 ? gb300::int8_plan_product(m, n, k, kept != 0, most)
                                        : gb300::int8_plan_gradient(kept, dtype, in_place != 0, vec != 0, m, n, k, most);
    const gb300::Int8TcForm form = gb300::int8_tc_form(p.shape);
    std::printf("%d %d %d %d %d %d %d %d %d %d %d\n", p.ok, p.small, int(p.shape), form.cols, form.run, p.a.splits, p.a.join,
                p.a.units, p.a.run, p.a.tiles_r, p.a.tiles_c);
  }
  return 0;
}
