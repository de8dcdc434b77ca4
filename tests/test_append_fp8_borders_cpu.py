"""The heads of test_append_fp8_borders_gpu.py decide what they are there for: evaluated in fp32 some of them get another scale, and
some values another code, than exactly."""
import numpy as np
import pytest

from oracle import served_layer as ref
from test_append_fp8_borders_gpu import CASES, EPS, exact, head, pairs


def in_fp32(x, w, pos, f, inter):
    F = np.float32
    y, (i, j) = x.astype(F), pairs(2 * len(f), inter)
    if w is not None:
        y = y * (F(1) / np.sqrt(np.sum(y * y, dtype=F) / F(len(x)) + F(EPS))) * w.astype(F)
    c, s = np.cos(pos * f).astype(F), np.sin(pos * f).astype(F)
    y[i], y[j] = y[i] * c - y[j] * s, y[i] * s + y[j] * c
    assert y.dtype == F
    return ref.pow2_codes(y.astype(np.float64))


@pytest.mark.parametrize("D,rot,inter,norm", CASES)
def test_heads_whose_codes_fp32_gets_wrong(D, rot, inter, norm):
    rng = np.random.default_rng(D + rot)
    scales = codes = above = 0
    for _ in range(24):
        x, w, pos, f = head(rng, D, rot, inter, norm)
        (y, e), (y32, e32) = exact(x, w, pos, f, inter), in_fp32(x, w, pos, f, inter)
        top = np.abs(ref.norm_rope(x[None, None], w, EPS, [pos], f, inter)[0]).max()
        step = top - 448.0 * 2.0 ** np.round(np.log2(top / 448.0))
        assert abs(step) <= 4 * 2.0 ** -23 * top  # the maximum is the one next to the border
        above += step > 0
        scales += e != e32
        codes += int((y != y32).sum()) if e == e32 else 0
    assert 4 <= above <= 20, above
    assert codes > 0 and scales > 0, (scales, codes)
