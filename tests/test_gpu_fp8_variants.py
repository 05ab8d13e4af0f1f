"""sgemm_fp8 on every kernel variant: each tile and cluster size, with each layout and
grouping of A and B.  A size stands for the variant that the plan takes for it; the test
asserts that it does, so that another rule cannot leave a variant untested.

Reference: the definition in 64 bits (on the GPU, from tables of the codes' values).
Error bound as in test_gpu_fp8_gemm.py: products of codes are exact, a block's 128 are
added in fp32, so |error| <= (128 + blocks + 16) * 2^-23 * sum |terms| and one rounding
to C's type.  Codes are of the formats' four largest binades, so that one wrong term
of a sum of some hundred shows."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp

pytestmark = pytest.mark.gpu

# group of B, tile rows, CTAs in a cluster, more tiles than CTAs: M, N, K
SIZES = {
    (1, 16, 1, False): (10, 62, 279), (1, 16, 1, True): (527, 1025, 261), (1, 16, 2, False): (281, 146, 1927),
    (1, 16, 4, False): (139, 129, 1314), (1, 16, 8, False): (10, 60, 1181), (1, 32, 1, False): (609, 390, 266),
    (1, 32, 1, True): (1027, 1045, 1009), (1, 32, 2, False): (274, 401, 4235), (1, 32, 4, False): (179, 258, 2823),
    (1, 32, 8, False): (139, 135, 5790), (1, 64, 1, False): (1233, 407, 393), (1, 64, 1, True): (99, 20913, 260),
    (1, 64, 2, False): (612, 385, 4633), (1, 64, 4, False): (375, 265, 3975), (1, 64, 8, False): (307, 133, 7765),
    (1, 128, 1, False): (105, 14747, 278), (1, 128, 1, True): (124, 29885, 267), (1, 128, 2, False): (705, 793, 8870),
    (1, 128, 4, False): (810, 274, 10588), (1, 256, 1, False): (813, 678, 291), (1, 256, 1, True): (2610, 1609, 274),
    (128, 16, 1, False): (9, 60, 263), (128, 16, 1, True): (1605, 333, 261), (128, 16, 2, False): (276, 142, 2404),
    (128, 16, 4, False): (159, 135, 1422), (128, 16, 8, False): (9, 60, 1290), (128, 32, 1, False): (807, 261, 266),
    (128, 32, 1, True): (78, 10476, 267), (128, 32, 2, False): (515, 431, 4275), (128, 32, 4, False): (274, 133, 2883),
    (128, 32, 8, False): (138, 142, 5770), (128, 64, 1, False): (690, 790, 761), (128, 64, 1, True): (98, 19701, 291),
    (128, 64, 2, False): (418, 665, 4257), (128, 64, 4, False): (356, 268, 4066), (128, 64, 8, False): (274, 142, 8062),
    (128, 128, 1, False): (108, 9892, 397), (128, 128, 1, True): (108, 29668, 279), (128, 128, 2, False): (812, 780, 9389),
    (128, 128, 4, False): (556, 394, 11115), (1, 128, 8, False): (2107, 60, 21247), (128, 128, 8, False): (479, 336, 22334),
    (128, 256, 1, False): (978, 514, 290), (128, 256, 1, True): (257, 9951, 260),
}
LAYOUTS = ["NT", "NN", "TN", "TT"]


def assert_plan(key):
    group, tile_m, ksplit, walks = key
    M, N, K = SIZES[key]
    tile_n = 256 if tile_m == 256 else 128
    assert sg.sgemm_fp8_plan(M, N, K, group) == (0, {"tile_m": tile_m, "tile_n": tile_n, "ksplit": ksplit})
    assert (-(-M // tile_m) * -(-N // tile_n) > (76 if tile_m == 256 else 152)) == walks
    return M, N, K


def _codes(gen, rows, cols, fmt, pad):
    """Codes, some of their rows starting off 16 bytes unless padded; the gaps hold NaN."""
    import torch
    ld = (cols + 15) // 16 * 16 if pad else cols
    low, high = (0x58, 0x7e) if fmt == "e4m3" else (0x6c, 0x7b)
    c = torch.randint(low, high + 1, (rows, ld), generator=gen, device="cuda", dtype=torch.uint8)
    c |= torch.randint(0, 2, (rows, ld), generator=gen, device="cuda", dtype=torch.uint8) << 7
    c[:, cols:] = 0x7f
    return c[:, :cols]


def _values(codes, scales, fmt, group, k_first):
    import torch
    rows, cols = codes.shape
    s, r, c = scales.double(), torch.arange(rows, device="cuda"), torch.arange(cols, device="cuda")
    v = torch.from_numpy(fp.TABLE[fmt]).cuda()[codes.long()]
    if group == 128:
        return v * s[(r // 128)[:, None], (c // 128)[None, :]]
    return v * (s[(r // 128)[:, None], c[None, :]] if k_first else s[(c // 128)[None, :], r[:, None]])


def _run(M, N, K, layout, ga, gb, fa, fb, ct, alpha, beta, pad, edit=None):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M * 7 + N * 3 + K)
    a = _codes(gen, *((M, K) if layout[0] == "N" else (K, M)), fa, pad)
    b = _codes(gen, *((K, N) if layout[1] == "N" else (N, K)), fb, pad)
    blocks = lambda n: -(-n // 128)  # noqa: E731

    def scales(mn, stored, group):
        shape = (blocks(K), mn) if group == 1 else tuple(blocks(n) for n in stored.shape)
        return torch.exp2(torch.rand(shape, generator=gen, device="cuda") * 8 - 6)

    sa, sb = scales(M, a, ga), scales(N, b, gb)
    if edit:
        edit(a if layout[0] == "N" else a.t(), b.t() if layout[1] == "N" else b, sa, sb)
    va = _values(a, sa, fa, ga, layout[0] == "T")
    vb = _values(b, sb, fb, gb, layout[1] == "N")
    va, vb = (va.t() if layout[0] == "T" else va), (vb.t() if layout[1] == "T" else vb)
    ctype = torch.float32 if ct == "f32" else torch.bfloat16
    full = torch.full((M + 2, N + 3), -3.0, device="cuda", dtype=ctype)
    C = full[1:-1, :N]
    C.copy_(torch.randn((M, N), generator=gen, device="cuda")) if beta else C.fill_(float("nan"))
    c0 = C.double()
    want = alpha * (va @ vb)
    size = abs(alpha) * (va.abs() @ vb.abs())
    if beta:
        want, size = want + beta * c0, size + (beta * c0).abs()
    dtype = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
    sg.fp8_gemm(a.view(dtype[fa]), sa, b.view(dtype[fb]), sb, C, *layout, alpha=alpha, beta=beta, a_group=ga, b_group=gb)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    got = C.double()
    assert bool((full[0] == -3).all()) and bool((full[-1] == -3).all()) and bool((full[:, N:] == -3).all())
    assert torch.equal(got.isnan(), want.isnan())
    odd = want.isinf()
    assert torch.equal(got[odd], want[odd]) and torch.equal(got.isinf(), odd)
    fine = want.isfinite()
    tol = (128 + blocks(K) + 16) * 2.0 ** -23 * size + (2.0 ** -24 if ct == "f32" else 2.0 ** -8) * want.abs()
    over = ((got - want).abs() / tol)[fine].max().item()
    assert over <= 1.0, over


@pytest.mark.parametrize("ga", [1, 128])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("key", SIZES)
def test_variant(key, layout, ga):
    M, N, K = assert_plan(key)
    i = list(SIZES).index(key) + LAYOUTS.index(layout)
    _run(M, N, K, layout, ga, key[0], "e4m3", ("e4m3", "e5m2")[i // 2 % 2], ("f32", "bf16")[i % 2],
         *((1.0, 0.0) if ga == 1 else (-1.5, 0.5)), pad=i % 4 < 2)


@pytest.mark.parametrize("key", [k for k in SIZES if not k[3]])
def test_special_values(key):
    """NaN, infinities, an infinity times zero, and a scale of zero, at the start and the end."""
    M, N, K = assert_plan(key)

    def edit(a, b, sa, sb):
        a[2, 5], a[M - 1, K - 1] = 0x7f, 0xff    # NaN
        a[3, 7], a[4, K - 2] = 0x7c, 0xfc        # infinities
        b[N - 1, 7] = 0x00                       # meets the first of them
        sa[0, 6] = 0.0                           # a row's first block

    for layout, beta in (("NT", 0.0), ("TN", 1.0)):
        _run(M, N, K, layout, 1, key[0], "e5m2", "e4m3", "f32", 1.0, beta, True, edit)
