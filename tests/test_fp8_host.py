"""Argument checks of the 8-bit entry points (no GPU: every case fails before
anything is launched), and the plain evaluation that the GPU tests compare
with, against closed forms."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


P = 1 << 20      # never dereferenced
F32, BF16, E4M3, E5M2 = sg.TYPE_F32, sg.TYPE_BF16, sg.TYPE_E4M3, sg.TYPE_E5M2


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({0: 2 ** 31}, -1), ({1: -1}, -2), ({1: 2 ** 31 - 1}, -2), ({2: 0}, -3),
    ({2: P + 2}, -3), ({3: E4M3}, -4), ({3: 9}, -4), ({4: 255}, -5), ({5: 2}, -6), ({6: 64}, -7),
    ({5: 1, 6: 1}, -7), ({7: 0}, -8), ({8: F32}, -9), ({9: 255}, -10), ({10: 0}, -11),
    ({10: P + 1}, -11), ({11: 9}, -12), ({5: 128, 6: 1, 11: 255}, -12), ({5: 128, 11: 1}, -12),
])
def test_quantize_refusals(change, want):
    args = [10, 256, P, F32, 256, 1, 128, P, E4M3, 256, P, 10]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_fp8_quantize(*args) == want


def test_quantize_of_nothing_is_ok():
    assert sg.sgemm_fp8_quantize(0, 5, 0, F32, 5, 1, 128, 0, E4M3, 5, 0, 1) == 0
    assert sg.sgemm_fp8_quantize(5, 0, 0, BF16, 1, 128, 128, 0, E5M2, 1, 0, 1) == 0


def test_formats():
    t = fp.TABLE["e4m3"]
    assert t[0x7e] == 448.0 and t[0x08] == 2.0 ** -6 and t[0x01] == 2.0 ** -9 and np.isnan(t[0xff])
    t = fp.TABLE["e5m2"]
    assert t[0x7b] == 57344.0 and t[0x04] == 2.0 ** -14 and t[0x01] == 2.0 ** -16 and t[0xfc] == -np.inf
    for f in ("e4m3", "e5m2"):
        v = fp.TABLE[f]
        ok = ~np.isnan(v)
        assert np.array_equal(fp.encode(v[ok], f), np.arange(256, dtype=np.uint8)[ok])


def test_formats_agree_with_torch():
    import torch
    c = torch.arange(256, dtype=torch.uint8)
    for f, d in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        assert np.array_equal(c.view(d).float().numpy().astype(np.float64), fp.TABLE[f], equal_nan=True)
        x = (torch.rand(4000, generator=torch.Generator().manual_seed(3)) - 0.5) * 2 * fp.LARGEST[f]
        assert np.array_equal(x.to(d).view(torch.uint8).numpy(), fp.encode(x.numpy(), f))


def test_plain_quantize_closed_form():
    x = np.zeros((2, 130), np.float32)
    x[0, 0], x[1, 129] = 896.0, -1.75
    codes, s = fp.quantize(x, (1, 128), "e4m3")
    assert s.shape == (2, 2) and s[0, 0] == 2.0 and s[1, 1] == np.float32(1.75) / np.float32(448)
    assert s[0, 1] == s[1, 0] == np.float32(2.0 ** -126)
    assert codes[0, 0] == 0x7e and codes[1, 129] == 0xfe and not codes[0, 1:].any()


@pytest.mark.parametrize("change,want", [
    ({0: "X"}, -1), ({1: "Q"}, -2), ({2: -1}, -3), ({3: 2 ** 31}, -4), ({4: -1}, -5), ({6: 0}, -7),
    ({7: F32}, -8), ({8: 299}, -9), ({9: 0}, -10), ({9: P + 2}, -10), ({10: 64}, -11), ({11: 9}, -12),
    ({10: 128, 11: 2}, -12), ({12: 0}, -13), ({13: BF16}, -14), ({14: 299}, -15), ({15: 0}, -16),
    ({16: 2}, -17), ({17: 2}, -18), ({16: 1, 17: 19}, -18), ({19: 0}, -20), ({19: P + 1}, -20),
    ({20: E4M3}, -21), ({21: 19}, -22), ({0: "T", 8: 9}, -9), ({1: "N", 14: 19}, -15),
])
def test_product_refusals(change, want):
    args = ["N", "T", 10, 20, 300, 1.0, P, E4M3, 300, P, 1, 10, P, E5M2, 300, P, 128, 3, 0.0, P, F32, 20]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_fp8(*args) == want


def test_product_of_nothing_is_ok():
    assert sg.sgemm_fp8("N", "T", 0, 20, 300, 1.0, 0, E4M3, 300, 0, 1, 1, 0, E4M3, 300, 0, 128, 3, 0.0, 0,
                        F32, 20) == 0


def test_product_plan_covers_every_shape():
    rng = np.random.default_rng(0)
    seen = set()
    for _ in range(3000):
        M, N, K = (int(np.exp(rng.uniform(0, np.log(20000)))) for _ in range(3))
        group = int(rng.choice([1, 128]))
        st, p = sg.sgemm_fp8_plan(M, N, K, group)
        nkb = -(-K // 128)
        assert st == 0 and 1 <= p["ksplit"] <= min(8, nkb)
        assert (p["tile_m"], p["tile_n"]) in {(16, 128), (32, 128), (64, 128), (128, 128), (256, 256)}
        tiles = -(-M // p["tile_m"]) * -(-N // p["tile_n"])
        if p["ksplit"] > 1:                     # clusters are resident at once
            assert p["tile_n"] == 128 and tiles * p["ksplit"] <= 152
        if p["tile_m"] > 16:
            assert p["tile_m"] < 2 * M
        seen.add((p["tile_m"], p["ksplit"] > 1))
    assert len(seen) == 9                       # every tile, the narrow ones with and without clusters
    for args, want in (((0, 1, 1), -1), ((1, 0, 1), -2), ((1, 1, 0), -3), ((1, 1, 1, 2), -4), ((1, 1, 1, 1, 0), -5)):
        assert sg.sgemm_fp8_plan(*args)[0] == want


def test_plain_product_closed_form():
    ones = np.full((3, 256), fp.encode(np.ones(1), "e4m3")[0])
    s = np.array([[2.0, 3.0, 4.0], [0.5, 0.25, 1.0]], np.float32)      # two blocks, three rows
    v = fp.values(ones, s, "e4m3", 1, False)
    out, size = fp.product(v, np.ones((256, 1)))
    assert out[:, 0].tolist() == [128 * 2.5, 128 * 3.25, 128 * 5.0] and np.array_equal(out, size)


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({0: 129}, -1), ({1: 0}, -2), ({2: 0}, -3), ({3: 0}, -4), ({3: 513}, -4), ({4: 0}, -5),
    ({4: 9}, -5), ({3: 64, 4: 17}, -5), ({5: 0}, -6), ({5: P + 1}, -6), ({6: E4M3}, -7), ({7: 255}, -8),
    ({8: P + 1}, -9), ({9: 0}, -10), ({10: 0}, -11), ({11: 0}, -12), ({12: 0}, -13), ({13: P + 2}, -14),
    ({14: 255}, -15), ({15: 128 * 256 - 1}, -16), ({16: 0}, -17), ({17: 0}, -18), ({18: 127}, -19),
    ({19: 1}, -20), ({21: 0}, -22), ({22: 255}, -23), ({23: 0}, -24), ({24: 0}, -25),
    ({10: P + 8}, sg.SGEMM_ERR_UNSUPPORTED), ({14: 257, 15: 257 * 128}, sg.SGEMM_ERR_UNSUPPORTED),
    ({19: 256 * 128 + 8}, sg.SGEMM_ERR_UNSUPPORTED),
])
def test_moe_refusals(change, want):
    args = [4, 256, 128, 8, 2, P, BF16, 256, P, P, P, P, P, P, 256, 256 * 128, P, P, 128, 256 * 128, 1, P, 256, P, P]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_moe(*args) == want


def test_moe_of_nothing_is_ok():
    assert sg.sgemm_moe(0, 256, 128, 8, 2, 0, F32, 256, 0, 0, 0, 0, 0, 0, 256, 256 * 128, 0, 0, 128, 256 * 128, 1,
                        0, 256, 0, 0) == 0


def test_plain_moe_closed_form():
    x = np.array([[2.0, 0.0]])
    gate, up, down = (np.array([[[a, 0.0]]]) for a in (1.0, 3.0, 0.0))
    down = np.array([[[5.0], [7.0]]])
    y, _, idx, w, _ = fp.moe(x, np.ones((1, 2)), gate, up, down, 1, False)
    h = 2 / (1 + np.exp(-2)) * 6
    assert np.allclose(y, [[5 * h, 7 * h]]) and w[0, 0] == 1.0 and idx[0, 0] == 0
