"""Host-side checks of the entry points for several new rows per sequence and of the 8-bit cache: every refusal happens
before the device is touched (these run without one); the oracle's own pins."""
import ctypes

import numpy as np
import pytest

from oracle import served_layer as ref
from test_served_layer_abi_cpu import BAD_CACHES, F, V, cache, caller  # noqa: F401


def cache8(V, **kw):
    d = dict(k=F, v=F, k_scales=F, v_scales=F, pages=F, n_pages=9, page_size=64, max_pages=7, Hkv=4, D=256)
    d.update(kw)
    return V.vp_paged_cache_fp8(*(d[n] for n in ("k", "v", "k_scales", "v_scales", "pages", "n_pages", "page_size", "max_pages", "Hkv", "D")))


def test_sizes(V):
    for size in (V.vp_prompt_attention_workspace_bytes, V.vp_paged_attention_rows_workspace_bytes):
        assert size(3, 100, 24, 4, 256) >= 256
        for bad in ((0, 100, 24, 4, 256), (65537, 100, 24, 4, 256), (3, 0, 24, 4, 256), (3, (1 << 24) + 1, 24, 4, 256),
                    (3, 100, 25, 4, 256), (3, 100, 2, 4, 256), (3, 100, 260, 4, 256), (3, 100, 24, 4, 96), (3, 100, 24, 0, 64),
                    (3, 100, 2048, 2048, 64), (3, 1 << 24, 128, 128, 64)):
            assert size(*bad) == 0, bad


def test_prompt_refusals(V):
    need = V.vp_prompt_attention_workspace_bytes(3, 100, 24, 4, 256)
    names = ["q", "ldq", "k", "ldk", "v", "ldv", "start", "S", "M", "Hq", "Hkv", "D", "scale", "gate", "out", "lse", "ws", "wb", "st"]
    call = caller(V.lib().vp_prompt_attention, names,
                  [F, 8192, F, 8192, F, 8192, F, 3, 100, 24, 4, 256, 0.0625, None, F, None, F, need, None])
    for name in ("q", "k", "v", "start", "out", "ws"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG, name
    for s in (float("nan"), float("inf"), 3e38, -3e38):
        assert call(scale=s) == V.VP_ERR_INVALID_ARG
    for kw in (dict(S=0), dict(S=65537), dict(M=0), dict(M=(1 << 24) + 1), dict(Hq=25), dict(Hq=2), dict(Hq=260), dict(D=96),
               dict(Hkv=0), dict(ldq=6136), dict(ldk=1016), dict(ldv=1016), dict(ldk=1 << 39), dict(ldq=1 << 39), dict(ldv=1 << 39)):
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(q=F + 8), dict(k=F + 8), dict(v=F + 8), dict(ldq=8196), dict(ldk=8196), dict(ldv=8196), dict(start=F + 2),
               dict(gate=F + 8), dict(out=F + 8), dict(lse=F + 2), dict(ws=F + 128)):
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw
    assert call(wb=need - 1) == V.VP_ERR_WORKSPACE


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_refusals(V, fp8):
    need = V.vp_paged_attention_rows_workspace_bytes(3, 100, 24, 4, 256)
    make = cache8 if fp8 else cache
    names = ["c", "q", "start", "len", "S", "M", "Hq", "scale", "gate", "out", "lse", "ws", "wb", "st"]
    call = caller(V.lib().vp_paged_attention_rows_fp8 if fp8 else V.lib().vp_paged_attention_rows, names,
                  [ctypes.byref(make(V)), F, F, F, 3, 100, 24, 0.0625, None, F, None, F, need, None])
    for name in ("c", "q", "len", "out", "ws"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG, name
    assert call(scale=float("nan")) == V.VP_ERR_INVALID_ARG
    for bad in BAD_CACHES:
        assert call(c=ctypes.byref(make(V, **bad))) == V.VP_ERR_SHAPE, bad
    for kw in (dict(S=0), dict(M=0), dict(Hq=25), dict(Hq=260), dict(Hq=2), dict(start=None)):  # M != S without row_start
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(q=F + 8), dict(start=F + 2), dict(len=F + 2), dict(gate=F + 8), dict(out=F + 8), dict(lse=F + 2), dict(ws=F + 128)):
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw
    assert call(wb=need - 1) == V.VP_ERR_WORKSPACE
    if fp8:
        for name in ("k", "v", "k_scales", "v_scales", "pages"):
            assert call(c=ctypes.byref(make(V, **{name: None}))) == V.VP_ERR_INVALID_ARG, name
        for name in ("k", "v", "k_scales", "v_scales"):
            assert call(c=ctypes.byref(make(V, **{name: F + 8}))) == V.VP_ERR_ALIGNMENT, name


def test_append_fp8_refusals(V):
    names = ["c", "q", "ldq", "k", "ldk", "v", "ldv", "qn", "kn", "eps", "rope", "start", "ctx", "S", "M", "Hq", "qo", "kvl", "stat", "st"]
    call = caller(V.lib().vp_paged_append_fp8, names,
                  [ctypes.byref(cache8(V)), F + 4096, 8192, F, 8192, F, 8192, None, None, 0.0, None, F, F, 3, 100, 24, F, None, None, None])
    for name in ("c", "k", "v", "ctx", "qo"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG, name
    for bad in BAD_CACHES:
        assert call(c=ctypes.byref(cache8(V, **bad))) == V.VP_ERR_SHAPE, bad
    assert call(c=ctypes.byref(cache8(V, k_scales=None))) == V.VP_ERR_INVALID_ARG
    assert call(c=ctypes.byref(cache8(V, v_scales=F + 4))) == V.VP_ERR_ALIGNMENT
    for kw in (dict(M=0), dict(S=0), dict(start=None), dict(ldk=1016), dict(ldq=6136)):
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(k=F + 8), dict(v=F + 8), dict(q=F + 4104), dict(qo=F + 8), dict(ldk=8196)):
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw


# ------------------------------------------------------------------ the oracle itself
def test_oracle_rows_attention_matches_torch():
    import torch
    rng = np.random.default_rng(0)
    k, v, q, g = (rng.standard_normal(s) for s in ((20, 2, 64), (20, 2, 64), (7, 4, 64), (7, 4, 64)))
    seen = np.arange(20)[None] <= 13 + np.arange(7)[:, None]
    out, mag, lse, dot = ref.rows_attention(q, [0, 7], [k], [v], [seen], 0.125, g)
    t = lambda x: torch.from_numpy(x).transpose(0, 1)  # noqa: E731
    kk, vv = t(k).repeat_interleave(2, 0), t(v).repeat_interleave(2, 0)
    want = torch.nn.functional.scaled_dot_product_attention(t(q), kk, vv, attn_mask=torch.from_numpy(seen), scale=0.125)
    assert np.allclose(out, (want.transpose(0, 1) * torch.sigmoid(torch.from_numpy(g))).numpy(), atol=1e-12)
    sc = (t(q) @ kk.transpose(1, 2) * 0.125).masked_fill(~torch.from_numpy(seen), -np.inf)
    assert np.allclose(lse, torch.logsumexp(sc, 2).T.numpy()) and (mag >= np.abs(out) - 1e-12).all() and (dot > 0).all()


def test_oracle_pow2_codes():
    y, e = ref.pow2_codes(np.array([[448.0, 1.0625, 3.0], [450.0, 0.0, 1.0], [0.0, 0.0, 0.0], [2.0 ** -130, 0.0, 0.0]]))
    assert e.tolist() == [0, 1, -118, -118] and y[0].tolist() == [448.0, 1.0, 3.0] and y[1].tolist() == [224.0, 0.0, 0.5]
    assert not y[2].any() and not y[3].any()
    import torch
    x = np.random.default_rng(1).standard_normal((50, 64)) * 100
    y, e = ref.pow2_codes(x)
    want = torch.from_numpy(x / 2.0 ** e[:, None]).float().to(torch.float8_e4m3fn).double().numpy()
    assert (y == want).mean() > 0.999 and (np.abs(x) / 2.0 ** e[:, None]).max() <= 448 and (np.abs(x).max(1) > 224 * 2.0 ** e).all()
