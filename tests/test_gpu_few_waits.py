"""The bounded waits of the 4-bit products run out where weights come from memory more slowly than a
warp takes them apart (one row of x): the call ends and says so, and the next one gives the
right result.  With more rows the weights may be there before every wait."""
import pytest

import dense_fp32_gemm_05_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("group,zeros,two", [(32, True, False), (64, False, True), (128, True, True), (128, False, False)])
@pytest.mark.parametrize("M", [1, 12, 40])
def test_waits_run_out(M, group, zeros, two, x):
    """90 MB of weights that are not in L2, three times."""
    import torch
    N, K = 20000, 9000
    gen = torch.Generator(device="cuda").manual_seed(M + group)
    q, s, z = sg.q4_quantize(torch.randn((N, K), device="cuda", generator=gen), group, not zeros)
    X = torch.randn((M, K), device="cuda", generator=gen).to(torch.bfloat16 if x == "bf16" else torch.float32)
    other = torch.empty(1 << 29, device="cuda", dtype=torch.uint8)
    more = dict(Q2=q, S2=s, Z2=z) if two else {}

    def call():
        other.zero_()
        return sg.q4_gemm(X, q, s, Z=z, group=group, **more)

    good, stream = call().clone(), torch.cuda.current_stream()
    assert sg.sgemm_device_error(stream) == 0
    seen = set()
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        for _ in range(3):
            call()
            seen.add(sg.sgemm_device_error(stream))
    finally:
        sg.sgemm_set_wait_limit(0)
    assert seen <= {0, sg.SGEMM_ERR_TIMEOUT}
    assert sg.SGEMM_ERR_TIMEOUT in seen or M > 1
    for _ in range(2):
        assert torch.equal(call(), good)
        assert sg.sgemm_device_error(stream) == 0
