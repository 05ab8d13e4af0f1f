"""The bounded waits of the feed-forward and 4-bit kernels: with a limit of 1 ns a role gives up
at its first wait for anything that is not there yet.  The call still ends, says so, and
leaves nothing behind: the next call gives the right result."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp

pytestmark = pytest.mark.gpu


def _check(call, sure=True):
    """call() -> tensors, the same every time.  sure: some of its waits are for what cannot be there."""
    import torch
    good = [t.clone() for t in call()]
    stream = torch.cuda.current_stream()
    assert sg.sgemm_device_error(stream) == 0
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        for _ in range(3):
            call()
            assert sg.sgemm_device_error(stream) in ((sg.SGEMM_ERR_TIMEOUT,) if sure else (0, sg.SGEMM_ERR_TIMEOUT))
    finally:
        sg.sgemm_set_wait_limit(0)
    for _ in range(2):
        again = call()
        assert sg.sgemm_device_error(stream) == 0
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(good, again))


# one of each tile: T, D, F
SIZES = [(100, 200, 500), (500, 600, 1500), (3000, 700, 2300)]


@pytest.mark.parametrize("T,D,F", SIZES)
def test_block(T, D, F):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, dy, gate, up, down = (fp.matrix(gen, *s, 0.2) for s in ((T, D), (T, D), (F, D), (F, D), (D, F)))
    _check(lambda: sg.ffn(x, gate, up, down)[:1])
    for keep in (torch.bfloat16, torch.float8_e4m3fn):
        kept = sg.ffn(x, gate, up, down, keep=keep)[1]
        _check(lambda: sg.ffn(x, gate, up, down, keep=keep)[1])
        _check(lambda: sg.ffn_backward(dy, x, gate, up, down, kept))


@pytest.mark.parametrize("M", [1, 12, 40])
@pytest.mark.parametrize("N,K", [(300, 5000), (20000, 300), (20000, 9000)])
def test_few_rows(M, N, K):
    """(4-bit weights may be there before every wait: x is laid out first, and taking codes apart
    lasts longer than their way from L2.)"""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M)
    q, s, z = sg.q4_quantize(torch.randn((N, K), device="cuda", generator=gen), 64, False)
    x = torch.randn((M, K), device="cuda", generator=gen).to(torch.bfloat16)
    _check(lambda: [sg.q4_gemm(x, q, s, Z=z, group=64)], False)


@pytest.mark.parametrize("T", [1, 12])
def test_block_of_few_tokens(T):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(T)
    for D, F in ((520, 2000), (5000, 9000)):
        x, gate, up, down = (fp.matrix(gen, *d, 0.1) for d in ((T, D), (F, D), (F, D), (D, F)))
        _check(lambda: sg.ffn(x, gate, up, down)[:1], D > 1000)
