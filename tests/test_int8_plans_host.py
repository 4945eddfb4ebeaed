"""Plans of the 8-bit integer operators' products (no GPU needed)."""
import os
import random
import subprocess

import pytest
import torch

import int8_plans

pytestmark = pytest.mark.skipif(not int8_plans.available(), reason="needs g++")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def sizes(rng, most):
    return max(1, int(2 ** rng.uniform(0, most)))


def test_accumulators_take_a_bounded_number_of_tokens():
    """The tensor core cuts off what is below an accumulator's last place, 6.5e-9 of a sum a token: at most 1/30 of half a step
    of a 16-bit result's type."""
    rng = random.Random(0)
    lines = [(1, t, out, t != 0, 1, sizes(rng, 22), sizes(rng, 14), sizes(rng, 14), *int8_plans.GB300)
             for t in range(3) for out in {t, 0} for _ in range(400)]
    for line, p in zip(lines, int8_plans.plans(lines)):
        out, tokens = line[2], line[5]
        most = {0: 512, 1: 16384, 2: 2048}[out]
        assert p.ok
        if p.small:
            taken = -(-tokens // (4 * 64)) * 64                     # a warp's share, in steps of 64 tokens
        else:
            share = -(-(-(-tokens // 128)) // p.splits) * 128
            taken = p.run_taken * 128 if p.run else share
            assert p.run == p.run_taken and (p.run == 0 or taken <= 2048)
        assert taken <= max(most, 512), (line, p)
        assert out == 0 or taken * 6.5e-9 <= {1: 2.0 ** -8, 2: 2.0 ** -11}[out] / 30


def test_plans_cover_the_product_once():
    rng = random.Random(1)
    lines = [(kind, rng.choice((0, 1, 2)), 0, 0, 1, sizes(rng, 16), sizes(rng, 15), sizes(rng, 16), *int8_plans.GB300)
             for kind in (0, 1) for _ in range(500)]
    for line, p in zip(lines, int8_plans.plans(lines)):
        m, n, k = line[5:8]
        if p.small:
            continue
        rows, cols, depth = (n, m, k) if line[0] == 0 else (k, n, m)
        assert p.tiles_r == -(-rows // 256) and p.tiles_c == -(-cols // p.cols)
        assert p.units == p.tiles_r * p.tiles_c * p.splits and 1 <= p.splits <= -(-depth // 128)
        if p.join:
            assert p.splits in (2, 4) and p.units // p.splits <= int8_plans.GB300[p.splits // 2]
        elif p.splits > 1:
            assert p.units <= int8_plans.GB300[0]


@pytest.mark.parametrize("size,kept,out,want", [
    ((16384, 4096, 4096), BF16, BF16, (256, 0)), ((16384, 4096, 4096), F16, F16, (256, 16)), ((4096, 4096, 1024), BF16, BF16, (256, 0)),
    ((32768, 4096, 4096), BF16, BF16, (256, 16)), ((16384, 4096, 4096), BF16, F32, (128, 4)), ((4096, 1024, 1024), F32, F32, (128, 4))])
def test_tiles_of_large_gradients(size, kept, out, want):
    p = int8_plans.gradient(*size, kept, out)
    assert not p.small and (p.cols, p.run) == want


def test_clusters_that_one_form_cannot_have_are_not_planned(tmp_path):
    """The counts that plans are made with are the least of all forms', a zero among them, whatever their order."""
    source = tmp_path / "least.cpp"
    source.write_text("""
        #include <cstdio>
        #include "int8_plan.h"
        int main() {
          for (int zero = 0; zero < 3; ++zero) {
            gb300::Int8LeastClusters least;
            for (int form = 0; form < 3; ++form) {
              least.take(1, 76 - form);
              least.take(2, form == zero ? 0 : 38 + form);
            }
            const gb300::Int8TcClusters n = least.clusters();
            std::printf("%d %d %d\\n", n.pairs, n.twos, n.fours);
          }
        }""")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    exe = str(tmp_path / "least")
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(int8_plans.ROOT, "dense_fp32_gemm_03_gb300", "csrc"), "-I",
                    os.path.join(int8_plans.ROOT, "include"), "-I", os.path.join(cuda, "include"), str(source), "-o", exe], check=True)
    assert subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")[:3] == ["74 0 0"] * 3


@pytest.mark.parametrize("clusters", [(76, 0, 18), (76, 38, 0), (76, 0, 0)])
def test_plans_without_some_clusters(clusters):
    for m, n, k in ((128, 4096, 4096), (4096, 1024, 1024), (1200, 520, 700)):
        for p in (int8_plans.product(m, n, k, clusters=clusters), int8_plans.gradient(m, n, k, BF16, clusters=clusters)):
            assert p.ok and (not p.join or clusters[p.splits // 2] > 0)
