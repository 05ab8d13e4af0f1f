"""sgemm_fp8 against the definition in 64 bits.

Error bound, from the arithmetic: products of codes are exact; a block's 128
products are added in fp32 (128 roundings or truncations, 2^-23 each at most,
of partial sums no larger than the sum of the magnitudes), a scale product, a
multiply-add for each block, up to 8 partial sums and the epilogue follow.  So
|error| <= (128 + blocks + 16) * 2^-23 * sum |terms|, and one rounding to C's
type (2^-24 or 2^-8 of the result)."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp

pytestmark = pytest.mark.gpu

CODE = {"e4m3": sg.TYPE_E4M3, "e5m2": sg.TYPE_E5M2}


def _codes(rng, rows, cols, fmt):
    return fp.encode(np.clip(rng.standard_normal((rows, cols)) * (fp.LARGEST[fmt] / 4),
                             -fp.LARGEST[fmt], fp.LARGEST[fmt]), fmt)


def _scales(rng, mn, k, k_first, group, stored):
    shape = (-(-k // 128), mn) if group == 1 else tuple(-(-n // 128) for n in stored)
    return np.exp2(rng.uniform(-6, 2, shape)).astype(np.float32)


def _dev(a, ld, off=0):
    """A device copy with leading dimension ld, `off` elements into its buffer; gaps hold a value that shows."""
    import torch
    rows, cols = a.shape
    buf = np.full(off + rows * ld + 16, 0x7f if a.dtype == np.uint8 else np.nan, dtype=a.dtype)
    buf[off: off + rows * ld].reshape(rows, ld)[:, :cols] = a
    t = torch.from_numpy(buf).cuda()
    return t, t.data_ptr() + off * a.itemsize


def _run(M, N, K, ta="N", tb="T", fa="e4m3", fb="e4m3", ga=1, gb=128, ct="f32", alpha=1.0, beta=0.0,
         pads=(0, 0, 0, 0, 0), offs=(0, 0, 0), seed=0, edit=None):
    import torch
    rng = np.random.default_rng(seed + M * 7 + N * 3 + K)
    sa_shape = (M, K) if ta == "N" else (K, M)
    sb_shape = (K, N) if tb == "N" else (N, K)
    a, b = _codes(rng, *sa_shape, fa), _codes(rng, *sb_shape, fb)
    sa = _scales(rng, M, K, ta == "T", ga, sa_shape)
    sb = _scales(rng, N, K, tb == "N", gb, sb_shape)
    if edit:
        edit(a, sa, b, sb)
    va, vb = fp.values(a, sa, fa, ga, ta == "T"), fp.values(b, sb, fb, gb, tb == "N")
    va, vb = (va.T if ta == "T" else va), (vb.T if tb == "T" else vb)
    c = rng.standard_normal((M, N)).astype(np.float32)
    ctype = torch.float32 if ct == "f32" else torch.bfloat16
    ldc = N + pads[4]
    bc = torch.full((M * ldc + 64 + offs[2],), -3.0, dtype=ctype, device="cuda")
    C = bc[32 + offs[2]: 32 + offs[2] + M * ldc].view(M, ldc)[:, :N]
    C.copy_(torch.from_numpy(c)) if beta != 0 else C.fill_(float("nan"))
    c0 = C.float().cpu().numpy().astype(np.float64)
    ha, pa = _dev(a, sa_shape[1] + pads[0], offs[0])
    hb, pb = _dev(b, sb_shape[1] + pads[1], offs[1])
    hsa, psa = _dev(sa, sa.shape[1] + pads[2])
    hsb, psb = _dev(sb, sb.shape[1] + pads[3])
    s = torch.cuda.current_stream()
    st = sg.sgemm_fp8(ta, tb, M, N, K, alpha, pa, CODE[fa], sa_shape[1] + pads[0], psa, ga,
                      sa.shape[1] + pads[2], pb, CODE[fb], sb_shape[1] + pads[1], psb, gb,
                      sb.shape[1] + pads[3], beta, C.data_ptr(),
                      sg.TYPE_F32 if ct == "f32" else sg.TYPE_BF16, ldc, s)
    assert st == 0
    assert sg.sgemm_device_error(s) == 0
    got = C.float().cpu().numpy().astype(np.float64)
    want, size = fp.product(va, vb, alpha, beta, c0 if beta != 0 else None)
    mask = torch.ones_like(bc, dtype=torch.bool)
    mask[32 + offs[2]: 32 + offs[2] + M * ldc].view(M, ldc)[:, :N] = False
    assert bool((bc[mask] == -3.0).all()), "written outside C"
    return got, want, size, -(-K // 128), ct


def _check(*args, **kw):
    got, want, size, nb, ct = _run(*args, **kw)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)])
    tol = (128 + nb + 16) * 2.0 ** -23 * size + (2.0 ** -24 if ct == "f32" else 2.0 ** -8) * np.abs(want) + 1e-37
    err = np.abs(got - want)[fine] / tol[fine]
    assert err.size == 0 or err.max() <= 1.0, err.max()
    return got


LAYOUTS = [("N", "T", 1, 128), ("N", "N", 1, 128), ("T", "N", 1, 1), ("T", "T", 128, 1), ("N", "T", 1, 1),
           ("T", "N", 128, 128)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 1, 1), (5, 200, 300), (16, 512, 2048), (17, 129, 130),
                                   (33, 640, 1000), (64, 256, 512), (100, 300, 400), (128, 128, 1024),
                                   (129, 257, 385), (300, 500, 700), (512, 384, 256)])
def test_layouts_and_sizes(layout, M, N, K):
    ta, tb, ga, gb = layout
    _check(M, N, K, ta, tb, ga=ga, gb=gb)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("layout", LAYOUTS[:3])
def test_code_types(fa, fb, layout):
    ta, tb, ga, gb = layout
    _check(70, 200, 333, ta, tb, fa, fb, ga, gb)


@pytest.mark.parametrize("ct", ["f32", "bf16"])
@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (-1.5, 0.5), (2.0, 0.0)])
@pytest.mark.parametrize("M,N,K", [(3, 200, 1500), (150, 270, 260)])
def test_epilogue(ct, alpha, beta, M, N, K):
    _check(M, N, K, ct=ct, alpha=alpha, beta=beta)


@pytest.mark.parametrize("layout", LAYOUTS[:4])
@pytest.mark.parametrize("pads,offs", [((16, 32, 3, 5, 7), (0, 0, 0)), ((1, 0, 0, 0, 0), (0, 0, 0)),
                                       ((0, 3, 0, 0, 1), (0, 0, 1)), ((0, 0, 0, 0, 0), (4, 0, 3)),
                                       ((8, 8, 0, 0, 0), (1, 13, 0))])
def test_strides_and_alignment(layout, pads, offs):
    ta, tb, ga, gb = layout
    _check(77, 208, 336, ta, tb, ga=ga, gb=gb, pads=pads, offs=offs)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 8192), (16, 1000, 8000), (2048, 1792, 256), (1500, 4100, 300),
                                   (4095, 3073, 129)])
def test_larger(M, N, K):
    _check(M, N, K, ct="bf16")


@pytest.mark.parametrize("layout", [("N", "T", 1, 128), ("T", "N", 1, 1)])
@pytest.mark.parametrize("shape", [(2700, 2600, 400), (2560, 2304, 1111)])
def test_many_tiles(layout, shape):
    ta, tb, ga, gb = layout
    _check(*shape, ta, tb, "e5m2", "e4m3", ga, gb)


@pytest.mark.parametrize("ct,alpha,beta", [("f32", 1.0, 1.0), ("f32", 0.5, 1.0), ("f32", 1.0, -2.0),
                                           ("bf16", 1.0, 1.0), ("bf16", 3.0, 0.0)])
@pytest.mark.parametrize("layout", [("N", "T", 1, 128), ("T", "N", 1, 1)])
@pytest.mark.parametrize("shape,pad,off", [((2560, 2304, 520), 0, 0), ((2500, 2312, 300), 4, 0),
                                           ((2500, 2309, 300), 0, 0), ((2500, 2308, 300), 0, 1)])
def test_wide_tiles_epilogue(ct, alpha, beta, layout, shape, pad, off):
    """Stores by TMA, additions by TMA, quads and single elements of C."""
    ta, tb, ga, gb = layout
    _check(*shape, ta, tb, "e4m3", "e5m2", ga, gb, ct, alpha, beta, pads=(0, 0, 0, 0, pad), offs=(0, 0, off))


def test_special_codes():
    def edit(a, sa, b, sb):
        a[2, 5] = 0x7f                # NaN (e5m2 code 0x7f too)
        a[3, 7] = 0x7c                # infinity
        a[4, 9] = 0xfc
        b[7, 11] = 0x00               # its product with the infinity of the same k: checked by class
        b[:, 7] = np.where(b[:, 7] & 0x7f, b[:, 7], 1)
        sa[0, 6] = 0.0
    _check(40, 160, 200, "N", "T", "e5m2", "e4m3", edit=edit)


def test_exact_small_integers():
    """Small integers: every sum is exact, so the result is the integer one."""
    import torch
    rng = np.random.default_rng(4)
    for M, N, K in ((9, 140, 500), (260, 300, 260)):
        a, b = rng.integers(-4, 5, (M, K)), rng.integers(-4, 5, (N, K))
        A = torch.from_numpy(a.astype(np.float32)).cuda().to(torch.float8_e4m3fn)
        B = torch.from_numpy(b.astype(np.float32)).cuda().to(torch.float8_e4m3fn)
        kb = -(-K // 128)
        SA = torch.full((kb, M), 2.0, device="cuda")
        SB = torch.full((-(-N // 128), kb), 0.25, device="cuda")
        C = torch.empty((M, N), device="cuda")
        sg.fp8_gemm(A, SA, B, SB, C)
        assert np.array_equal(C.cpu().numpy().astype(np.float64), 0.5 * (a @ b.T))


def test_no_product_term():
    import torch
    for ct in (torch.float32, torch.bfloat16):
        C = torch.randn(30, 50, device="cuda").to(ct)
        want = (C.float() * 0.5).to(ct)
        A, B = (torch.zeros(n, 64, device="cuda").to(torch.float8_e4m3fn) for n in (30, 50))
        SA, SB = torch.ones(1, 30, device="cuda"), torch.ones(1, 1, device="cuda")
        sg.fp8_gemm(A, SA, B, SB, C, alpha=0.0, beta=0.5)
        assert torch.equal(C, want)
        C.fill_(float("nan"))
        E = torch.empty(30, 0, device="cuda", dtype=torch.float8_e4m3fn)
        F = torch.empty(50, 0, device="cuda", dtype=torch.float8_e4m3fn)
        sg.fp8_gemm(E, torch.empty(0, 30, device="cuda"), F, torch.empty(1, 0, device="cuda"), C)
        assert not C.any()


def test_same_result_every_time_and_on_another_stream():
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((24, 4096), generator=g, device="cuda")
    w = torch.randn((1000, 4096), generator=g, device="cuda")
    qx, sx = sg.fp8_quantize(x)
    qw, sw = sg.fp8_quantize(w, (128, 128))
    outs = [sg.fp8_gemm(qx, sx, qw, sw, torch.empty(24, 1000, device="cuda")) for _ in range(5)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs.append(sg.fp8_gemm(qx, sx, qw, sw, torch.empty(24, 1000, device="cuda")))
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0], o) for o in outs[1:])
    assert sg.sgemm_device_error() == 0
    # and it is the product of the quantised values
    ref = x.double() @ w.double().t()
    rel = (outs[0].double() - ref).norm() / ref.norm()
    assert rel < 0.06          # two roundings to 4 significant bits, 2^-4 at most each, independent


def test_linear_layer_gradients_against_differences():
    """loss = <y, dy>, y = x W^T of the quantised values: its derivatives by central
    differences of the 64-bit loss, and by the two backward products."""
    import torch
    T, D, N = 40, 160, 130
    g = torch.Generator(device="cuda").manual_seed(8)
    x, w, dy = (torch.randn(s, generator=g, device="cuda") for s in ((T, D), (N, D), (T, N)))
    qw, sw = sg.fp8_quantize(w, (128, 128))
    qdy, sdy = sg.fp8_quantize(dy, (1, 128), torch.float8_e5m2)
    dx = sg.fp8_gemm(qdy, sdy, qw, sw, torch.empty(T, D, device="cuda"), "N", "N")
    qdyt, sdyt = sg.fp8_quantize(dy, (128, 1), torch.float8_e5m2)
    qxt, sxt = sg.fp8_quantize(x, (128, 1))
    dw = sg.fp8_gemm(qdyt, sdyt, qxt, sxt, torch.zeros(N, D, device="cuda"), "T", "N", beta=1.0, b_group=1)
    val = lambda q, s, f, grp, kf: fp.values(q.view(torch.uint8).cpu().numpy(), s.cpu().numpy(), f, grp, kf)  # noqa: E731
    W, G1 = val(qw, sw, "e4m3", 128, False), val(qdy, sdy, "e5m2", 1, False)
    X, G2 = val(qxt, sxt, "e4m3", 1, True), val(qdyt, sdyt, "e5m2", 1, True)
    rng = np.random.default_rng(1)
    for _ in range(10):
        i, j = rng.integers(T), rng.integers(D)
        step = np.zeros((T, D)); step[i, j] = 0.5
        x0 = x.double().cpu().numpy()
        diff = (((x0 + step) @ W.T * G1).sum() - ((x0 - step) @ W.T * G1).sum())
        assert abs(diff - dx[i, j].item()) <= 1e-5 * (np.abs(G1[i]) @ np.abs(W[:, j])) + 1e-9 * abs(
            (np.abs(x0) @ np.abs(W.T) * np.abs(G1)).sum())
        n, d = rng.integers(N), rng.integers(D)
        step = np.zeros((N, D)); step[n, d] = 0.5
        diff = ((X @ (W + step).T * G2).sum() - (X @ (W - step).T * G2).sum())
        assert abs(diff - dw[n, d].item()) <= 1e-5 * (np.abs(G2[:, n]) @ np.abs(X[:, d])) + 1e-9 * abs(
            (np.abs(X) @ np.abs(W.T) * np.abs(G2)).sum())


def test_a_wait_that_runs_out_is_reported():
    """The bounded waits: a limit of 1 ns makes a role give up; the call still ends, and says so."""
    import torch
    x, w = torch.randn(200, 8192, device="cuda"), torch.randn(300, 8192, device="cuda")
    qx, sx = sg.fp8_quantize(x)
    qw, sw = sg.fp8_quantize(w, (128, 128))
    C = torch.empty(200, 300, device="cuda")
    good = sg.fp8_gemm(qx, sx, qw, sw, torch.empty_like(C))
    torch.cuda.synchronize()
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        sg.fp8_gemm(qx, sx, qw, sw, C)
        assert sg.sgemm_device_error(torch.cuda.current_stream()) == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_set_wait_limit(0)
    sg.fp8_gemm(qx, sx, qw, sw, C)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    assert torch.equal(C, good)
