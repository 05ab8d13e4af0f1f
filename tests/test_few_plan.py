"""How the products of few rows are cut (few_plan, compiled with the host compiler): what the GPU tests'
sizes are for, and that what a cut counts on fits the GPU."""
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
# clusters of 1 .. 8 CTAs that a GB300 holds, with two CTAs an SM and with one (as it was asked)
HELD = [[304, 152, 97, 74, 58, 46, 38, 36], [152, 76, 46, 36, 28, 23, 15, 15]]


@pytest.fixture(scope="module")
def cuts(tmp_path_factory):
    from dense_fp32_gemm_05_gb300 import build
    include = os.path.join(os.path.dirname(os.path.dirname(shutil.which(build.nvcc()) or build.nvcc())), "include")
    out = str(tmp_path_factory.mktemp("few_plan") / "few_plan_host")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-isystem", include, os.path.join(HERE, "few_plan_host.cpp"), "-o", out],
                   check=True, timeout=300)

    def run(sizes):
        r = subprocess.run([out] + [str(n) for h in HELD for n in h], input="\n".join(" ".join(map(str, s)) for s in sizes),
                           capture_output=True, text=True, timeout=60, check=True)
        lines = [dict(zip(("nt", "wk", "ks", "depth", "ring", "bytes"), map(int, t.split()))) for t in r.stdout.splitlines()]
        assert len(lines) == len(sizes)
        return lines
    return run


def _ctas(size, cut):
    """CTAs (clusters, where the sum is cut) of a call, all blocks of rows of x together."""
    M, N, K, group, f32, gated = size
    per_cta = (16 if gated else 32) * (8 // cut["wk"])
    per_block = 8 * cut["nt"] // (2 if f32 and group else 1)
    return -(-N // per_cta) * -(-M // per_block)


def test_sizes_of_the_gpu_tests(cuts):
    """Sums cut over 3, 6, 5 and 7 CTAs, and calls of more CTAs than the GPU holds, as
    test_clusters_of_any_size and test_few_tokens_in_clusters_of_three take them."""
    sizes = {(1, 24000, 768, 64, 0, 0): 3, (4, 11776, 1536, 64, 0, 0): 6, (1, 14848, 1280, 64, 0, 0): 5, (4, 9728, 1792, 64, 0, 0): 7,
             (4, 12032, 768, 64, 0, 1): 3, (30, 11700, 768, 64, 0, 0): 3, (1, 40000, 300, 64, 0, 0): 1, (1, 80000, 520, 64, 0, 0): 1,
             (5, 12032, 192, 0, 0, 1): 3}
    assert [c["ks"] for c in cuts(list(sizes))] == list(sizes.values())
    wide = (1, 80000, 520, 64, 0, 0)
    assert _ctas(wide, cuts([wide])[0]) > HELD[0][0]


def test_blocks_of_rows_count(cuts):
    """Rows of x past a block's take CTAs of their own: what is cut runs together with them."""
    for size in ((33, 4096, 8192, 128, 1, 0), (64, 4096, 8192, 128, 1, 0), (64, 2048, 4096, 64, 1, 0), (100, 1024, 8192, 128, 0, 0),
                 (70, 4096, 2048, 64, 0, 1), (200, 2048, 4096, 128, 0, 0)):
        cut = cuts([size])[0]
        assert _ctas(size, cut) <= HELD[1][cut["ks"] - 1], (size, cut)


def test_every_cut_runs_together_and_fits(cuts):
    rng = random.Random(0)
    sizes = [(int(2 ** rng.uniform(0, 10)), int(2 ** rng.uniform(0, 17)), int(2 ** rng.uniform(0, 16)), rng.choice((32, 64, 128)),
              rng.randrange(2), rng.randrange(2)) for _ in range(4000)]
    sizes += [(rng.randrange(1, 17), *s[1:3], 0, 0, s[5]) for s in sizes[:1000]]
    seen = set()
    for size, cut in zip(sizes, cuts(sizes)):
        M, N, K, group, f32, gated = size
        stages = -(-K // (256 if group else 64))
        assert 1 <= cut["ring"] <= 2 and 1 <= cut["depth"] <= stages and cut["bytes"] + 1024 <= 225 * 1024, (size, cut)
        assert cut["ks"] <= stages
        if (cut["wk"], cut["ks"]) != (1, 1):
            assert _ctas(size, cut) <= HELD[cut["nt"] > 2][cut["ks"] - 1], (size, cut)
        seen.add((cut["nt"], cut["ks"]))
    assert {k for n, k in seen if n <= 2} == set(range(1, 9)) and {k for n, k in seen if n > 2} == {1, 2, 3, 4}
