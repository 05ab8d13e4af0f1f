"""How near 8-bit parts come to an activation: the split that sgemm_moe's documentation
states (scale the block by a power of two, round to E4M3, times 32 what is left, again),
evaluated with numpy, against the stated bounds."""
import numpy as np
import pytest

from tests import fp8_plain as fp


def split(v, parts):
    """The sum of the parts of a block's values."""
    scale = 2.0 ** (7 - np.floor(np.log2(np.abs(v).max())))
    y, out = v * scale, np.zeros(v.shape)
    for i in range(parts):
        q = fp.decode(fp.encode(y, "e4m3"), "e4m3")
        out += q / 32.0 ** i
        y = (y - q) * 32
    return out / scale


def _blocks():
    rng = np.random.default_rng(0)
    for n in range(200):
        v = rng.standard_normal(128) * np.exp2(rng.uniform(-30, 0, 128) * (n % 4) / 3)
        if n % 5 == 0:
            v[7] = 2.0 ** 18                    # one value far above the others
        yield v.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("parts,of_value,of_largest", [(4, 19, 32), (3, 14, 27), (2, 9, 22)])
def test_bounds(parts, of_value, of_largest):
    """Each value to the larger of two bounds: 2^-19 (14, 9) of it, 2^-32 (27, 22) of the block's largest."""
    worst = 0.0
    for v in _blocks():
        err = np.abs(split(v, parts) - v)
        bound = np.maximum(np.abs(v) * 2.0 ** -of_value, np.abs(v).max() * 2.0 ** -of_largest)
        assert np.all(err <= bound)
        worst = max(worst, (err / bound).max())
    assert worst > 0.4                          # (and no bound is far off)


def test_bf16_in_two_parts():
    """Exact down to 2^-14 of the block's largest, the rest to 2^-22 of it."""
    for v in _blocks():
        v = (v.astype(np.float32).view(np.uint32) & 0xffff0000).view(np.float32).astype(np.float64)
        err, most = np.abs(split(v, 2) - v), np.abs(v).max()
        assert not err[np.abs(v) >= 2.0 ** -14 * most].any()
        assert err.max() <= 2.0 ** -22 * most
