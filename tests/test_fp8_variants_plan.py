"""The sizes that test_gpu_fp8_variants.py takes for sgemm_fp8's variants, against the
rule that picks them (no GPU)."""
import random

import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests.test_gpu_fp8_variants import SIZES, assert_plan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


@pytest.mark.parametrize("key", SIZES)
def test_sizes_take_their_variant(key):
    assert_plan(key)


def test_every_variant_has_a_size():
    """Every tile and cluster size that the rule takes over a wide range of sizes."""
    rng, seen = random.Random(0), set()
    for _ in range(60000):
        M, N, K = (int(2 ** rng.uniform(0, 14.5)) for _ in range(3))
        group = rng.choice((1, 128))
        plan = sg.sgemm_fp8_plan(M, N, K, group)[1]
        seen.add((group, plan["tile_m"], plan["ksplit"]))
    assert seen == {k[:3] for k in SIZES}
