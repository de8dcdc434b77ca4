"""Keys of vp_paged_append_fp8 whose exact values, after norm and rotation, lie within a few fp32 steps of where the answer changes: the
head's maximum of 448 * 2^e, every other value of a tie between two codes.  An evaluation in fp32 gets a part of them wrong
(test_append_fp8_borders_cpu.py); the codes and scales have to be the exact values', all of them."""
import numpy as np
import pytest
import torch

from oracle import served_layer as ref
from test_rows_attention_gpu import Cache, codes_equal
from test_served_layer_gpu import f32, freqs, i32

pytestmark = pytest.mark.gpu

EPS = 1e-6
CASES = [(64, 0, False, True), (64, 64, True, True), (64, 32, False, True), (128, 128, False, True), (128, 96, True, True),
         (256, 64, True, True), (256, 256, False, True), (64, 64, False, False), (128, 32, True, False), (256, 256, True, False),
         (256, 128, False, False)]


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


def to_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def step32(x):
    return np.ldexp(1.0, np.frexp(np.abs(x))[1] - 24)


def near(rng, x, steps=4):
    """x and up to `steps` fp32 steps more or less."""
    return x + rng.uniform(-steps, steps, np.shape(x)) * step32(x)


def pairs(rot, inter):
    i = np.arange(rot // 2) * 2 if inter else np.arange(rot // 2)
    return i, i + 1 if inter else i + rot // 2


def head(rng, D, rot, inter, norm):
    """One key x [D] (bf16 values), its weights (fp32 values or None), position and frequencies."""
    e = int(rng.integers(-9, -5))
    ties = (rng.integers(8, 16, D) + 0.5) / 8 * np.exp2(rng.integers(0, 8, D) + e)  # below 256 * 2^e
    top = int(rng.integers(0, D if norm else rot // 2))
    i, j = pairs(rot, inter)
    if norm:
        y = near(rng, ties) * rng.choice([-1.0, 1.0], D)
        y[top] = near(rng, 448.0 * 2.0 ** e, 0.75)
        x = to_bf16(rng.uniform(0.3, 3.0, D) * rng.choice([-1.0, 1.0], D))
        pos, f = int(rng.integers(0, 32)), np.array(freqs(rot) if rot else [])
        c, s = np.cos(pos * f), np.sin(pos * f)
        y[i], y[j] = y[i] * c + y[j] * s, y[j] * c - y[i] * s  # before the rotation
        w = y / (x / np.sqrt((x * x).mean() + np.float64(np.float32(EPS))))
        return x, w.astype(np.float32).astype(np.float64), pos, f
    # no weights to choose: the angles, at position 1
    x = to_bf16(rng.uniform(0.1, 2.0, D) * 2.0 ** (e + 6))
    x[i[top]], x[j[top]] = 8 * 2.0 ** (e + 6), 3 * 2.0 ** (e + 6)
    r, phi = np.hypot(x[i], x[j]), np.arctan2(x[j], x[i])
    want = near(rng, np.where(ties[:rot // 2] < r, ties[:rot // 2], np.ldexp(1.0625, np.frexp(r)[1] - 2)))
    want[top] = near(rng, 448.0 * 2.0 ** e, 0.75)
    return x, None, 1, np.mod(np.arccos(want / r) - phi, 2 * np.pi)


def exact(x, w, pos, f, inter):
    y, _ = ref.norm_rope(x[None, None], w, EPS, [pos], f, inter)
    return ref.pow2_codes(y[0, 0])


@pytest.mark.parametrize("copies", [1, 700])
@pytest.mark.parametrize("D,rot,inter,norm", CASES)
def test_append_fp8_next_to_borders_and_ties(V, D, rot, inter, norm, copies):
    """copies: one row, or many rows per call, whose blocks take several heads per group of lanes; the second head is the
    first one's negative."""
    rng, P, Hkv = np.random.default_rng(D + rot), 16, 2
    c = Cache(V, 1, copies, 2, P, Hkv, D, True)
    for n in range(24 if copies == 1 else 6):
        x, w, pos, f = head(rng, D, rot, inter, norm)
        y, e = exact(x, w, pos, f, inter)
        k = torch.from_numpy(np.tile(np.stack([x, -x]), (copies, 1, 1))).to(torch.bfloat16).cuda()
        V.vp_paged_append_fp8(c.desc(), None, 0, k, Hkv * D, k, Hkv * D, None, None if w is None else f32(w), EPS,
                              V.vp_rope(list(f), inter) if rot else None, None, i32([pos] * copies), copies, copies, 0, None)
        pg = torch.from_numpy(c.table[:, pos // P]).cuda().long()
        got, sc = c.k[pg, :, pos % P].cpu().numpy(), c.ks[pg, :, pos % P].cpu().numpy().astype(int) - 127
        assert (sc == e).all(), (n, sc[0], e)
        assert codes_equal(got[:, 0], np.tile(y, (copies, 1))) and codes_equal(got[:, 1], np.tile(-y, (copies, 1))), n
