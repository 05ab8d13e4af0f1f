"""The 8-bit kernels' bounded waits, on every kind of tile: with a limit of 1 ns a role
gives up at its first wait for anything that is not there yet.  The call still ends, says
so, and leaves nothing behind: the next call gives the right result."""
import pytest

import dense_fp32_gemm_05_gb300 as sg

pytestmark = pytest.mark.gpu

NARROW = [  # M, N, K, groups of B, tile rows, CTAs in a cluster
    (16, 2000, 4000, 128, 16, 8), (400, 1500, 200, 128, 16, 1), (300, 130, 3000, 128, 32, 4),
    (70, 10000, 100, 128, 32, 1), (300, 130, 8000, 128, 64, 8), (100, 6000, 100, 128, 64, 1),
    (673, 818, 9611, 128, 128, 2), (104, 10016, 411, 128, 128, 1),
    (300, 130, 2000, 1, 16, 2), (127, 10000, 100, 1, 32, 1), (400, 300, 4000, 1, 64, 4), (117, 10621, 393, 1, 128, 1)]


def _run(M, N, K, group, layout="NT"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    ta, tb = layout
    shape = lambda n, along: (n, K) if along else (K, n)  # noqa: E731
    group_of = lambda n, along: (128, 128) if n == 128 else (1, 128) if along else (128, 1)  # noqa: E731
    qx, sx = sg.fp8_quantize(torch.randn(shape(M, ta == "N"), generator=g, device="cuda"), group_of(1, ta == "N"))
    qw, sw = sg.fp8_quantize(torch.randn(shape(N, tb == "T"), generator=g, device="cuda"), group_of(group, tb == "T"))
    C = torch.empty((M, N), device="cuda")
    call = lambda: sg.fp8_gemm(qx, sx, qw, sw, C, ta, tb, b_group=group)  # noqa: E731
    good = call().clone()
    stream = torch.cuda.current_stream()
    assert sg.sgemm_device_error(stream) == 0
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        for _ in range(3):
            call()
            assert sg.sgemm_device_error(stream) == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_set_wait_limit(0)
    for _ in range(2):
        C.fill_(float("nan"))
        call()
        assert sg.sgemm_device_error(stream) == 0
        assert torch.equal(C, good)


@pytest.mark.parametrize("M,N,K,group,tile_m,ksplit", NARROW)
def test_narrow_tiles(M, N, K, group, tile_m, ksplit):
    plan = {"tile_m": tile_m, "tile_n": 128, "ksplit": ksplit}
    assert sg.sgemm_fp8_plan(M, N, K, group) == (0, plan)
    _run(M, N, K, group)


WIDE = [  # M, N, K, layout, groups of B
    (400, 1500, 100, "NT", 128), (2000, 1900, 2000, "NT", 128), (2500, 2300, 700, "NN", 128),
    (2000, 1900, 2000, "TN", 1), (3000, 2300, 700, "TN", 1), (2000, 300, 100, "NT", 1)]


@pytest.mark.parametrize("M,N,K,layout,group", WIDE)
def test_wide_tiles(M, N, K, layout, group):
    """Tiles on pairs of SMs: what either has under way when a role gives up lands before they leave."""
    plan = {"tile_m": 256, "tile_n": 256, "ksplit": 1}
    assert sg.sgemm_fp8_plan(M, N, K, group) == (0, plan)
    _run(M, N, K, group, layout)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,topk", [(1, 8, 2), (12, 8, 2), (40, 8, 4), (100, 5, 3)])
def test_layer(dtype, T, E, topk):
    """The layer with 8, 16, 32 and 64 columns for an expert."""
    import torch
    from tests.test_gpu_moe import Layer, _x
    layer = Layer(640, 320, E, seed=T)
    x, stream = _x(T, 640, dtype), torch.cuda.current_stream()
    good = layer.run(x, topk, True)[0].clone()
    assert sg.sgemm_device_error(stream) == 0
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        for _ in range(3):
            layer.run(x, topk, True)
            assert sg.sgemm_device_error(stream) == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_set_wait_limit(0)
    for _ in range(2):
        assert torch.equal(layer.run(x, topk, True)[0], good)
        assert sg.sgemm_device_error(stream) == 0
