"""Host-side checks of the served attention layer's entry points: every refusal happens before the
device is touched (these run without one), and the descriptors' sizes."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import served_layer as ref

F = 0x10000000  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import build
    build()
    from weight_streaming_gb300 import _lib
    return _lib


def caller(fn, names, ok):
    def call(**kw):
        a = list(ok)
        for key, val in kw.items():
            a[names.index(key)] = val
        return fn(*a)
    return call


def test_quant_refusals(V):
    call = caller(V.lib().vp_quant_fp8, ["x", "t", "ld", "M", "K", "q", "s", "st"], [F, 0, 256, 4, 256, F, F, None])
    for name in ("x", "q", "s"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG
    assert call(t=2) == V.VP_ERR_INVALID_ARG and call(t=-1) == V.VP_ERR_INVALID_ARG
    for kw in (dict(M=0), dict(M=-1), dict(M=(1 << 24) + 1), dict(K=0), dict(K=8), dict(K=250), dict(K=65552, ld=65552),
               dict(ld=248)):
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    assert call(x=F + 8) == V.VP_ERR_ALIGNMENT and call(q=F + 8) == V.VP_ERR_ALIGNMENT
    assert call(s=F + 2) == V.VP_ERR_ALIGNMENT
    assert call(ld=260) == V.VP_ERR_ALIGNMENT and call(t=1, ld=258) == V.VP_ERR_ALIGNMENT


def test_add_rmsnorm_refusals(V):
    names = ["x", "t", "ld", "res", "w", "eps", "M", "K", "h", "q", "s", "st"]
    call = caller(V.lib().vp_add_rmsnorm_fp8, names, [F, 0, 512, F, F, 1e-6, 4, 256, F, F, F, None])
    for name in ("x", "q", "s"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG
    for eps in (0.0, -1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == V.VP_ERR_INVALID_ARG
    # in place on x only as a dense bf16 matrix
    assert call(h=F, x=F, ld=512) == V.VP_ERR_INVALID_ARG and call(t=1, ld=256) == V.VP_ERR_INVALID_ARG
    G = F + 4096
    assert call(x=G, K=16400, ld=16400) == V.VP_ERR_SHAPE and call(x=G, K=24) == V.VP_ERR_SHAPE
    assert call(x=G, res=F + 8) == V.VP_ERR_ALIGNMENT and call(x=G, w=F + 2) == V.VP_ERR_ALIGNMENT
    assert call(x=G, h=F + 8) == V.VP_ERR_ALIGNMENT


def test_linear_block_sizes_and_refusals(V):
    assert V.vp_packed_bytes_fp8_block(5120, 17408) == 5120 * 17408
    assert V.vp_packed_bytes_fp8_block(144, 272) == 256 * 384  # padded to whole 128 x 128 tiles
    for N, K in ((0, 256), (8, 256), (24, 256), (256, 8), (256, 65552), ((1 << 20) + 16, 256)):
        assert V.vp_packed_bytes_fp8_block(N, K) == 0
        assert V.vp_linear_fp8_block_workspace_bytes(1, N, K) == 0
    assert V.vp_linear_fp8_block_workspace_bytes(0, 256, 256) == 0
    assert V.vp_linear_fp8_block_workspace_bytes((1 << 20) + 1, 256, 256) == 0
    need = V.vp_linear_fp8_block_workspace_bytes(4, 256, 256)
    assert need >= 256
    L = V.lib()
    pk = caller(L.vp_pack_fp8_block, ["w", "N", "K", "p", "pb", "st"], [F, 256, 256, F, 65536, None])
    assert pk(w=None) == V.VP_ERR_INVALID_ARG and pk(p=None) == V.VP_ERR_INVALID_ARG
    assert pk(pb=65535) == V.VP_ERR_INVALID_ARG and pk(N=250) == V.VP_ERR_SHAPE
    assert pk(w=F + 8) == V.VP_ERR_ALIGNMENT and pk(p=F + 8) == V.VP_ERR_ALIGNMENT
    names = ["w", "ws", "x", "xs", "y", "t", "M", "N", "K", "wsp", "wb", "st"]
    call = caller(L.vp_linear_fp8_block, names, [F, F, F, F, F, 0, 4, 256, 256, F, need, None])
    for name in ("w", "ws", "x", "xs", "y", "wsp"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG
    assert call(t=2) == V.VP_ERR_INVALID_ARG
    for kw in (dict(M=0), dict(M=(1 << 20) + 1), dict(N=250), dict(K=250), dict(K=65552), dict(N=1 << 20, K=65536, M=0)):
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(w=F + 8), dict(ws=F + 2), dict(x=F + 8), dict(xs=F + 2), dict(y=F + 8), dict(wsp=F + 128)):
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw
    assert call(wb=need - 1) == V.VP_ERR_WORKSPACE


def cache(V, **kw):
    a = dict(k=F, v=F, pages=F, n_pages=100, page_size=64, max_pages=10, Hkv=4, D=256)
    a.update(kw)
    return V.vp_paged_cache(**a)


BAD_CACHES = [dict(D=96), dict(D=512), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(Hkv=0),
              dict(Hkv=1025), dict(n_pages=0), dict(max_pages=0), dict(n_pages=1 << 24), dict(max_pages=1 << 25)]


def test_paged_append_refusals(V):
    names = ["c", "q", "ldq", "k", "ldk", "v", "ldv", "qn", "kn", "eps", "rope", "rs", "ctx", "S", "M", "Hq", "out", "len",
             "status", "st"]
    rope = V.vp_rope([1.0] * 128, True)
    ok = [ctypes.byref(cache(V)), F, 6144, F, 1024, F, 1024, None, None, 0.0, ctypes.byref(rope), F, F, 4, 4, 24, F, None,
          None, None]
    call = caller(V.lib().vp_paged_append, names, ok)
    for name in ("c", "k", "v", "ctx", "out"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG, name
    assert call(len=F) == V.VP_ERR_INVALID_ARG  # kv_len may not be ctx itself
    for field in ("k", "v", "pages"):
        assert call(c=ctypes.byref(cache(V, **{field: None}))) == V.VP_ERR_INVALID_ARG
        assert call(c=ctypes.byref(cache(V, **{field: F + 2}))) == V.VP_ERR_ALIGNMENT
    for bad in BAD_CACHES:
        assert call(c=ctypes.byref(cache(V, **bad))) == V.VP_ERR_SHAPE, bad
    assert call(qn=F) == V.VP_ERR_INVALID_ARG and call(kn=F, eps=float("nan")) == V.VP_ERR_INVALID_ARG
    assert call(out=F, q=F, ldq=8192) == V.VP_ERR_INVALID_ARG  # in place only when dense
    for kw in (dict(M=0), dict(S=0), dict(S=65537), dict(M=(1 << 24) + 1), dict(Hq=0), dict(Hq=4097), dict(ldq=6136),
               dict(ldk=1016), dict(ldv=1016), dict(rs=None, M=5)):
        kw.setdefault("q", F + 4096)
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(q=F + 8), dict(k=F + 8), dict(v=F + 8), dict(ldk=1028), dict(ldv=1028), dict(ldq=6148), dict(rs=F + 2),
               dict(ctx=F + 2), dict(len=F + 2), dict(status=F + 2), dict(qn=F + 2, eps=1e-6), dict(out=F + 8)):
        kw.setdefault("q", F + 4096)
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw
    for r, want in ((V.vp_rope([1.0] * 4, True), V.VP_ERR_SHAPE), (V.vp_rope([1.0] * 136, True), V.VP_ERR_SHAPE),
                    (V.vp_rope([float("nan")] * 8, False), V.VP_ERR_INVALID_ARG),
                    (V.vp_rope([float("inf")] * 8, False), V.VP_ERR_INVALID_ARG)):
        assert call(rope=ctypes.byref(r)) == want
    r = V.vp_rope([1.0] * 8, True)
    r.inv_freq = None
    assert call(rope=ctypes.byref(r)) == V.VP_ERR_INVALID_ARG
    r.inv_freq, r.rot_dim = F, -16
    assert call(rope=ctypes.byref(r)) == V.VP_ERR_SHAPE


def test_paged_attention_sizes_and_refusals(V):
    need = V.vp_paged_attention_workspace_bytes(4, 24, 4, 256)
    assert need >= 256
    for S, Hq, Hkv, D in ((0, 24, 4, 256), (8193, 24, 4, 256), (4, 25, 4, 256), (4, 2, 4, 256), (4, 68, 4, 256),
                          (4, 24, 4, 96), (4, 24, 0, 256), (8192, 9, 9, 64)):
        assert V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D) == 0, (S, Hq, Hkv, D)
    names = ["c", "q", "len", "S", "Hq", "scale", "gate", "out", "lse", "ws", "wb", "st"]
    call = caller(V.lib().vp_paged_attention, names,
                  [ctypes.byref(cache(V)), F, F, 4, 24, 0.0625, None, F, None, F, need, None])
    for name in ("c", "q", "len", "out", "ws"):
        assert call(**{name: None}) == V.VP_ERR_INVALID_ARG, name
    assert call(scale=float("nan")) == V.VP_ERR_INVALID_ARG and call(scale=float("inf")) == V.VP_ERR_INVALID_ARG
    assert call(scale=3e38) == V.VP_ERR_INVALID_ARG  # times log2 e
    for bad in BAD_CACHES:
        assert call(c=ctypes.byref(cache(V, **bad))) == V.VP_ERR_SHAPE, bad
    for kw in (dict(S=0), dict(S=8193), dict(Hq=25), dict(Hq=68), dict(Hq=2)):
        assert call(**kw) == V.VP_ERR_SHAPE, kw
    for kw in (dict(q=F + 8), dict(len=F + 2), dict(gate=F + 8), dict(out=F + 8), dict(lse=F + 2), dict(ws=F + 128)):
        assert call(**kw) == V.VP_ERR_ALIGNMENT, kw
    assert call(wb=need - 1) == V.VP_ERR_WORKSPACE


# ------------------------------------------------------------------ the oracle itself
def test_oracle_e4m3_matches_torch():
    import torch
    c = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_value(c), want, equal_nan=True)
    assert np.array_equal(np.signbit(ref.e4m3_value(c)), np.signbit(want))


def test_oracle_rope_turns_and_linear_by_hand():
    """A quarter turn exchanges a pair; block scales multiply their own block only."""
    x = np.arange(1.0, 33.0).reshape(1, 1, 32)
    for inter in (True, False):
        y, mag = ref.norm_rope(x, None, 0.0, [1], [np.pi / 2] * 8, inter)
        i = np.arange(8) * 2 if inter else np.arange(8)
        j = i + 1 if inter else i + 8
        assert np.allclose(y[0, 0, i], -x[0, 0, j], atol=1e-12) and np.allclose(y[0, 0, j], x[0, 0, i], atol=1e-12)
        assert np.array_equal(y[0, 0, 16:], x[0, 0, 16:])
    xq, wq = np.full((1, 144), 0x38, np.uint8), np.full((144, 144), 0x38, np.uint8)  # 1.0 everywhere
    y, a = ref.linear_block(xq, [[2.0, 3.0]], wq, [[1.0, 10.0], [5.0, 100.0]])
    assert y[0, 0] == 128 * 2 + 16 * 30 and y[0, 143] == 128 * 10 + 16 * 300 and np.array_equal(y, a)


def test_oracle_paged_attention_matches_torch():
    import torch
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((5, 2, 16, 64)), rng.standard_normal((5, 2, 16, 64))
    q = rng.standard_normal((2, 4, 64))
    pages = np.array([[3, 1], [4, 0]], np.int32)
    out, mag, lse, dot = ref.paged_attention(q, k, v, pages, [20, 0], 0.125)
    kk = torch.from_numpy(np.concatenate([k[3], k[1]], 1)[:, :20]).repeat_interleave(2, 0)
    vv = torch.from_numpy(np.concatenate([v[3], v[1]], 1)[:, :20]).repeat_interleave(2, 0)
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[0])[:, None], kk, vv, scale=0.125)[:, 0]
    assert np.allclose(out[0], want.numpy(), atol=1e-12) and not out[1].any() and np.all(np.isinf(lse[1]))
    assert np.allclose(lse[0], torch.logsumexp((torch.from_numpy(q[0])[:, None] * kk).sum(-1) * 0.125, 1).numpy())


def test_oracle_add_rmsnorm_matches_torch():
    import torch
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 272)).astype(np.float32)
    res = oracle.bf16_round(rng.standard_normal((3, 272)))
    w = rng.standard_normal(272)
    h, y = ref.add_rmsnorm(x, res, w, 1e-6)
    r = torch.from_numpy(res.view(np.int16).copy()).view(torch.bfloat16)
    want_h = (torch.from_numpy(x) + r.float()).to(torch.bfloat16)
    assert np.array_equal(h.view(np.int16), want_h.view(torch.int16).numpy())
    want = torch.nn.functional.rms_norm(want_h.double(), (272,), torch.from_numpy(w), float(np.float32(1e-6)))
    assert np.allclose(y, want.numpy(), rtol=1e-12)
    assert np.allclose(ref.block_scales(y)[:, 2], np.abs(y[:, 256:]).max(1) / 448)
