"""sgemm_fp8 writes C inside its M x N window and nowhere else, whatever the window's
place in its rows."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b_group", [1, 128])
@pytest.mark.parametrize("ctype,beta", [(torch.float32, 0.0), (torch.float32, 1.0), (torch.bfloat16, 0.0),
                                        (torch.bfloat16, 1.0)])
@pytest.mark.parametrize("columns,gap", [(1600, 16), (1601, 15), (1603, 13), (1604, 12), (1607, 9), (1615, 1), (1629, 19)])
def test_gap_after_the_last_column(b_group, ctype, beta, columns, gap):
    """Wide tiles, rows of C on 16 bytes: stored by TMA (beta = 0) or added by it (fp32, beta = 1).
    The gap holds -0.0, so that an addition of zero shows too."""
    M, N, K = 2000, columns, 256
    assert sg.sgemm_fp8_plan(M, N, K, b_group)[1]["tile_m"] == 256
    assert (N + gap) * (4 if ctype == torch.float32 else 2) % 16 == 0
    gen = torch.Generator(device="cuda").manual_seed(N)
    a, b = (torch.randint(-3, 4, (n, K), generator=gen, device="cuda").float() for n in (M, N))
    A, B = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    SA = torch.ones(K // 128, M, device="cuda")
    SB = torch.ones(K // 128, N, device="cuda") if b_group == 1 else torch.ones(-(-N // 128), K // 128, device="cuda")
    full = torch.full((M + 16, N + gap), -0.0, device="cuda", dtype=ctype)
    C = full[8: 8 + M, :N]
    C.fill_(2.0)
    sg.fp8_gemm(A, SA, B, SB, C, beta=beta, b_group=b_group)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    want = torch.full_like(full, -0.0)
    want[8: 8 + M, :N] = (a @ b.t() + 2.0 * beta).to(ctype)       # integers: every sum is exact
    same = torch.int32 if ctype == torch.float32 else torch.int16
    outside = torch.ones_like(full, dtype=torch.bool)
    outside[8: 8 + M, :N] = False
    assert torch.equal(full.view(same)[outside], want.view(same)[outside]), "written outside C"
    assert torch.equal(C, want[8: 8 + M, :N])


@pytest.mark.parametrize("b_group", [1, 128])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("exponent", [-140, -130, -128])
def test_additions_keep_subnormal_numbers(b_group, offset, exponent):
    """alpha = beta = 1 in fp32 below the normal numbers: C on 16 bytes is added to by TMA, C off them
    by fused multiply-adds.  Sums and C are integers times 2^exponent and 2^-149, so both are exact."""
    M, N, K = 2000, 1600, 256
    assert sg.sgemm_fp8_plan(M, N, K, b_group)[1]["tile_m"] == 256
    gen = torch.Generator(device="cuda").manual_seed(3)
    a, b = (torch.randint(-2, 3, (n, K), generator=gen, device="cuda").float() for n in (M, N))
    a[:100] = 0                                                    # (a product of zero: C stays as it is)
    A, B = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    SA = torch.full((K // 128, M), 2.0 ** -60, device="cuda")
    SB = torch.full((K // 128, N) if b_group == 1 else (-(-N // 128), K // 128), 2.0 ** (exponent + 60), device="cuda")
    buf = torch.empty(M * N + 4, device="cuda")
    C = buf[offset: offset + M * N].view(M, N)
    C.copy_((torch.randint(-(1 << 20), 1 << 20, (M, N), generator=gen, device="cuda").double() * 2.0 ** -149).float())
    assert bool(((C != 0) & (C.abs() < 2.0 ** -126)).any())
    want = (C.double() + (a.double() @ b.double().t()) * 2.0 ** exponent).float()
    sg.fp8_gemm(A, SA, B, SB, C, beta=1.0, b_group=b_group)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    assert torch.equal(C, want)
