"""GPU parity of the attention of several new rows per sequence (vp_prompt_attention, vp_paged_attention_rows,
vp_paged_attention_rows_fp8) and of the 8-bit cache's append (vp_paged_append_fp8) against the fp64 definitions in
oracle/served_layer.py, through the C ABI.

Tolerances, with u = 2^-24 (half an fp32 step) and bf16's half step 2^-8:
  scores     D products, exact in fp32, and D additions at 2 u each (the tensor core may cut): 2 D u of scale * sum |q k| =: e,
             the same for the common factor log2 e and the subtraction (4 u of the score, itself below sum |q k| scale).
  outputs    weights exp(2 e) - 1, their rounding to bf16 (2^-8), the exponential (2^-22), up to n additions at 2 u and n in the
             divisor at u: times sum p |v|; division and gate 16 u; then the output's half step.
  lse        2 e, 2^-20 for exponential and logarithm, n u for the sum, 4 u of itself.
  append     the codes are the exact value's: equal, but for values that fp64 itself cannot tell from a tie."""
import math

import numpy as np
import pytest
import torch

from helpers import workspace
from oracle import served_layer as ref
from test_served_layer_gpu import U, assert_within, bf16, f32, f64, freqs, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


class Cache:
    """Random cached keys and values (bf16, or codes and scales), each (sequence, page) on a page of its own."""

    def __init__(self, V, seed, S, max_pages, P, Hkv, D, fp8, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.V, self.S, self.P, self.Hkv, self.D, self.max_pages, self.fp8 = V, S, P, Hkv, D, max_pages, fp8
        self.n = S * max_pages + spare
        shape = (self.n, Hkv, P, D)
        if fp8:
            self.k, self.v = ((100.0 * torch.randn(shape, generator=g, device="cuda")).clamp_(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8) for _ in "kv")
            self.ks, self.vs = (torch.randint(118, 122, shape[:3], generator=g, device="cuda", dtype=torch.uint8) for _ in "kv")
        else:
            self.k, self.v = (torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16) for _ in "kv")
        self.table = np.random.default_rng(seed).permutation(self.n)[:S * max_pages].reshape(S, max_pages).astype(np.int32)
        self.pages = i32(self.table)

    def desc(self):
        if self.fp8:
            return self.V.vp_paged_cache_fp8(self.k, self.v, self.ks, self.vs, self.pages, self.n, self.P, self.max_pages,
                                             self.Hkv, self.D)
        return self.V.vp_paged_cache(self.k, self.v, self.pages, self.n, self.P, self.max_pages, self.Hkv, self.D)

    def values(self, s, n):
        """fp64 keys and values [n][Hkv][D] of sequence s, and which positions exist."""
        t = np.arange(n)
        pg = self.table[s][t // self.P]
        there = (pg >= 0) & (pg < self.n)
        at = torch.from_numpy(np.where(there, pg, 0)).cuda().long(), torch.from_numpy(t % self.P).cuda()
        out = []
        for x, sc in ((self.k, getattr(self, "ks", None)), (self.v, getattr(self, "vs", None))):
            y = x[at[0], :, at[1]]
            if self.fp8:
                e = sc[at[0], :, at[1]].double().cpu().numpy()
                out.append(ref.e4m3_value(y.cpu().numpy()) * np.where(e == 255, np.nan, 2.0 ** (e - 127))[..., None])
            else:
                out.append(f64(y))
        return out[0], out[1], there

    def attend(self, q, start, kv_len, M, Hq, scale, gate, out, lse, ws, S=None, stream=None):
        f = self.V.vp_paged_attention_rows_fp8 if self.fp8 else self.V.vp_paged_attention_rows
        f(self.desc(), q, start, kv_len, S or self.S, M, Hq, scale, gate, out, lse, ws, stream)


def want_of(q, start, keys, values, ctx, there, scale, gate):
    seen = []
    for s in range(len(start) - 1):
        n, L = start[s + 1] - start[s], 0 if keys[s] is None else len(keys[s])
        ok = np.arange(L)[None] <= ctx[s] + np.arange(n)[:, None]
        seen.append(ok if there is None else ok & there[s][None])
    return ref.rows_attention(f64(q), start, keys, values, seen, scale, None if gate is None else f64(gate)), max(
        [1] + [len(k) for k in keys if k is not None])


def check(out, lse, want, n, D, what):
    o, mag, l, dot = want
    e = (2 * D * U + 4 * U) * dot
    bound = mag * (np.exp(2 * e)[..., None] - 1 + 2.0 ** -8 + 2.0 ** -22 + 3 * n * U + 16 * U) + 2.0 ** -8 * np.abs(o) + 1e-37
    assert_within(f64(out), o, bound, what + " out")
    if lse is not None:
        got, some = f64(lse), np.isfinite(l)
        assert np.array_equal(np.isneginf(got), ~some), what + " lse"
        assert_within(got[some], l[some], (2 * e + 2.0 ** -20 + n * U + 4 * U * np.abs(np.where(some, l, 0)))[some], what + " lse")


def buffers(M, Hq, D, gate, seed=5):
    rng = np.random.default_rng(seed)
    return (torch.full((M, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((M, Hq), 7.0, device="cuda"),
            bf16(rng, (M, Hq, D), 2.0) if gate else None)


# ------------------------------------------------------------------ whole prompts
@pytest.mark.parametrize("D,Hq,Hkv,rows,gate,scale", [
    (64, 1, 1, [1], False, None), (128, 4, 2, [2, 0, 1], True, None), (256, 24, 4, [63, 1, 126], True, None),
    (64, 16, 2, [129, 128, 127], False, None), (128, 32, 8, [257, 1, 600], True, 0.2), (256, 6, 1, [700], False, -0.07),
    (128, 3, 3, [391, 0, 0, 5], False, 0.0), (64, 64, 1, [70], False, None), (256, 64, 1, [33, 2], True, None),
    (256, 5, 5, [300, 17], False, None), (128, 14, 2, [1000], False, None), (256, 2, 2, [1100], True, None),
])
def test_prompt(V, D, Hq, Hkv, rows, gate, scale):
    rng = np.random.default_rng(sum(rows) + D)
    scale = D ** -0.5 if scale is None else scale
    start = np.cumsum([2] + rows)  # rows 0 and 1 are padding, and so are the last two
    M, S, ld = start[-1] + 2, len(rows), (Hq + 2 * Hkv) * D + 24
    x = bf16(rng, (M, ld), 1.3)
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]
    out, lse, g = buffers(M, Hq, D, gate)
    ws = workspace(V.vp_prompt_attention_workspace_bytes(S, M, Hq, Hkv, D))
    V.vp_prompt_attention(q, ld, k, ld, v, ld, i32(start), S, M, Hq, Hkv, D, scale, g, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    for t in (out[:2], out[-2:], lse[:2], lse[-2:]):
        assert bool((t == 7.0).all())  # padding rows
    part = [slice(a, b) for a, b in zip(start, start[1:])]
    keys, values = ([f64(t[p]).reshape(-1, Hkv, D) for p in part] for t in (k, v))
    want, n = want_of(q.reshape(M, Hq, D), start, keys, values, [0] * S, None, scale, g)
    inner = slice(2, M - 2)
    check(out[inner], lse[inner], [w[inner] for w in want], n, D, "prompt")


# ------------------------------------------------------------------ rows over a paged cache
ROWS = [
    (64, 2, 1, 16, [1], [0], False), (128, 4, 2, 16, [5, 1], [11, 127], True), (256, 24, 4, 64, [8] * 4, [0, 63, 700, 1500], True),
    (128, 32, 8, 16, [1] * 7, [0, 15, 16, 127, 128, 129, 900], False), (256, 24, 4, 64, [1] * 3, [2999, 5, 64], True),
    (64, 16, 2, 128, [1, 40, 0, 3], [500, 3, 77, 1000], False), (128, 16, 1, 32, [2, 2], [400, 31], False),
    (256, 4, 1, 128, [9], [2000], False), (64, 8, 8, 32, [33, 300], [64, 65], True), (128, 8, 2, 64, [200, 1], [0, 850], False),
    (256, 6, 2, 16, [90, 150], [10, 333], True), (128, 64, 1, 128, [3, 5], [130, 0], False), (256, 8, 4, 32, [17, 1, 128], [600, 1, 0], True),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,P,rows,ctx,gate", ROWS)
def test_rows(V, D, Hq, Hkv, P, rows, ctx, gate, fp8):
    S, L = len(rows), [a + b for a, b in zip(rows, ctx)]
    c = Cache(V, D + P, S, -(-max(L) // P) + 1, P, Hkv, D, fp8)
    start = np.cumsum([1] + rows)
    M = start[-1] + 1
    q = bf16(np.random.default_rng(P), (M, Hq, D), 1.5)
    out, lse, g = buffers(M, Hq, D, gate)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(start), i32(L), M, Hq, D ** -0.5, g, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    for t in (out[0], out[-1], lse[0], lse[-1]):
        assert bool((t == 7.0).all())
    kv = [c.values(s, L[s]) for s in range(S)]
    want, n = want_of(q, start, [x[0] for x in kv], [x[1] for x in kv], ctx, None, D ** -0.5, g)
    inner = slice(1, M - 1)
    check(out[inner], lse[inner], [w[inner] for w in want], n, D, f"rows {D} {fp8}")
    # again, and without lse: the same bits
    again = torch.full_like(out, 7.0)
    c.attend(q, i32(start), i32(L), M, Hq, D ** -0.5, g, again, None, ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    if rows == [1] * S:  # one row per sequence without row_start
        one = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda")
        c.attend(q[1:1 + S].contiguous(), None, i32(L), S, Hq, D ** -0.5, None if g is None else g[1:1 + S].contiguous(), one, None, ws)
        assert torch.equal(one.view(torch.int16), out[inner].view(torch.int16))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,n,ctx", [(256, 6, 1, 1, 40000), (128, 4, 1, 8, 30000), (64, 2, 1, 300, 20000), (256, 2, 1, 200, 9000)])
def test_rows_cut_along_long_contexts(V, D, Hq, Hkv, n, ctx, fp8):
    c = Cache(V, 3, 1, -(-(n + ctx) // 64), 64, Hkv, D, fp8)
    q = bf16(np.random.default_rng(1), (n, Hq, D), 1.5)
    out, lse, g = buffers(n, Hq, D, True)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, n, Hq, Hkv, D))
    c.attend(q, i32([0, n]), i32([n + ctx]), n, Hq, D ** -0.5, g, out, lse, ws)
    k, v, _ = c.values(0, n + ctx)
    want, m = want_of(q, [0, n], [k], [v], [ctx], None, D ** -0.5, g)
    check(out, lse, want, m, D, "cut")


def test_rows_many_sequences_and_shared_pages(V):
    """Thousands of short sequences over the same few pages (the prompt that they share)."""
    S, Hq, Hkv, D, P = 5000, 4, 2, 64, 16
    c = Cache(V, 9, 1, 6, P, Hkv, D, False)
    rng = np.random.default_rng(2)
    c.S, c.max_pages = S, 2
    c.table = rng.integers(0, c.n, (S, 2)).astype(np.int32)
    c.pages = i32(c.table)
    rows = rng.integers(0, 3, S)
    L = rows + rng.integers(0, 2 * P - 2, S)
    start = np.concatenate([[0], np.cumsum(rows)])
    M = int(start[-1])
    q = bf16(rng, (M, Hq, D), 1.5)
    out, lse, _ = buffers(M, Hq, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(start), i32(L), M, Hq, 0.125, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    kf, vf = f64(c.k), f64(c.v)
    keys, values = ([x[c.table[s, np.arange(L[s]) // P], :, np.arange(L[s]) % P] for s in range(S)] for x in (kf, vf))
    want, n = want_of(q, start, keys, values, L - rows, None, 0.125, None)
    check(out, lse, want, n, D, "many")


# ------------------------------------------------------------------ what rows do not see
@pytest.mark.parametrize("D,Hq,Hkv,n", [(64, 4, 2, 200), (128, 2, 1, 300), (256, 4, 1, 150), (256, 2, 1, 20), (128, 4, 1, 7)])
def test_values_that_a_row_does_not_see_have_no_effect(V, D, Hq, Hkv, n):
    rng = np.random.default_rng(D)
    q, k, v = bf16(rng, (n, Hq, D)), bf16(rng, (n, Hkv, D)), bf16(rng, (n, Hkv, D))
    ws = workspace(V.vp_prompt_attention_workspace_bytes(2, n, Hq, Hkv, D))
    run = lambda k, v, start: (lambda o: (V.vp_prompt_attention(q, Hq * D, k, Hkv * D, v, Hkv * D, i32(start), len(start) - 1, n,  # noqa: E731
                                          Hq, Hkv, D, 0.1, None, o, None, ws), o)[1])(torch.empty_like(q))
    good, cut = run(k, v, [0, n]), n // 2
    k2, v2 = k.clone(), v.clone()
    bad = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda").to(torch.bfloat16)
    k2[cut:] = bad[torch.randint(0, 3, k2[cut:].shape, device="cuda")]
    v2[cut:] = bad[torch.randint(0, 3, v2[cut:].shape, device="cuda")]
    got = run(k2, v2, [0, n])
    assert torch.equal(got[:cut], good[:cut])
    # behind a sequence lies the next one
    first = run(k, v, [0, cut])
    assert torch.equal(run(k2, v2, [0, cut])[:cut], first[:cut])
    # a value that is none reaches its column, of the rows that see it and the heads that share it
    v3 = v.clone()
    v3[cut, 0, 3], v3[cut + 1, Hkv - 1, D - 1] = float("nan"), float("inf")
    got, G = run(k, v3, [0, n]).float(), Hq // Hkv
    clean = torch.ones_like(got, dtype=torch.bool)
    clean[cut:, :G, 3] = False
    clean[cut + 1:, Hq - G:, D - 1] = False
    assert torch.equal(got[clean], good.float()[clean]) and not bool(torch.isfinite(got[~clean]).any())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,n,L", [(128, 1, 70), (256, 3, 201), (64, 40, 130), (256, 150, 333)])
def test_what_lies_behind_the_end_has_no_effect(V, D, n, L, fp8):
    P, Hq, Hkv = 32, 2, 1
    c = Cache(V, 4, 1, -(-L // P) + 2, P, Hkv, D, fp8)
    q = bf16(np.random.default_rng(1), (n, Hq, D))
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, n, Hq, Hkv, D))
    res = []
    for _ in range(2):
        out = torch.empty_like(q)
        c.attend(q, i32([0, n]), i32([L]), n, Hq, 0.1, None, out, None, ws)
        res.append(out)
        for t in range(L, c.max_pages * P):
            pg, sl = int(c.table[0, t // P]), t % P
            c.k[pg, :, sl] = c.v[pg, :, sl] = 0x7F if fp8 else float("nan")
            if fp8:
                c.ks[pg, :, sl] = c.vs[pg, :, sl] = 255
    assert torch.equal(res[0], res[1])
    assert V.vp_read_status(ws) == V.VP_OK


def test_scales_from_the_smallest_to_the_largest(V):
    """Every scale byte of the format's range: code * 2^(scale - 127) as a value, 255 as NaN in the columns that see it."""
    D, Hq, P, L = 64, 1, 128, 256
    c = Cache(V, 6, 1, 2, P, 1, D, True)
    c.ks[:] = 120
    q = bf16(np.random.default_rng(1), (1, Hq, D), 1e-3)  # about even weights
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, 1, Hq, 1, D))
    for e in (9, 60, 119, 134, 135, 200, 240):
        c.vs[:] = e
        out = torch.empty_like(q)
        c.attend(q, None, i32([L]), 1, Hq, 1.0, None, out, None, ws, S=1)
        k, v, _ = c.values(0, L)
        want, n = want_of(q, [0, 1], [k], [v], [L - 1], None, 1.0, None)
        check(out, None, want, n, D, f"scale {e}")
    c.vs[int(c.table[0, 0]), 0, 5] = 255
    c.attend(q, None, i32([L]), 1, Hq, 1.0, None, out, None, ws, S=1)
    assert bool(torch.isnan(out).all())


def test_scores_of_minus_infinity(V):
    """Rows all of whose scores are -infinity give zeros; a key of -infinity beside others has no weight."""
    n, Hq, D = 140, 2, 128
    rng = np.random.default_rng(3)
    q, k, v = bf16(rng, (n, Hq, D)).abs_(), bf16(rng, (n, 1, D)), bf16(rng, (n, 1, D))
    k[:100] = float("-inf")
    out, lse, _ = buffers(n, Hq, D, False)
    ws = workspace(V.vp_prompt_attention_workspace_bytes(1, n, Hq, 1, D))
    V.vp_prompt_attention(q, Hq * D, k, D, v, D, i32([0, n]), 1, n, Hq, 1, D, 0.1, None, out, lse, ws)
    assert not bool(out[:100].any()) and bool(torch.isneginf(lse[:100]).all())
    seen = np.tril(np.ones((n, n), bool))
    seen[:, :100] = False
    kk = f64(k).copy()
    kk[:100] = 0.0
    want = ref.rows_attention(f64(q), [0, n], [kk], [f64(v)], [seen], 0.1)
    check(out, lse, want, n, D, "-inf")


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_lengths_and_pages(V, fp8):
    P, Hq, Hkv, D, S = 16, 4, 2, 128, 6
    rows, L = [3, 40, 2, 1, 5, 2], [50, 20, 97, -1, 5, 64]  # too short, behind the table, negative
    c = Cache(V, 8, S, 6, P, Hkv, D, fp8)
    c.table[0, 1], c.table[5, 0], c.table[5, 1], c.table[5, 2], c.table[5, 3] = -1, c.n, 1 << 30, -(1 << 31), c.n + 5
    c.pages = i32(c.table)
    start = np.cumsum([0] + rows)
    M = int(start[-1])
    q = bf16(np.random.default_rng(1), (M, Hq, D))
    out, lse, _ = buffers(M, Hq, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(start), i32(L), M, Hq, 0.1, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
    ok = [0, 4, 5]
    kv = {s: c.values(s, L[s]) for s in ok}
    keys, values = ([kv[s][i] if s in kv else None for s in range(S)] for i in (0, 1))
    there = [kv[s][2] if s in kv else None for s in range(S)]
    seen = [np.zeros((rows[s], 0), bool) if s not in kv else
            (np.arange(L[s])[None] <= L[s] - rows[s] + np.arange(rows[s])[:, None]) & there[s][None] for s in range(S)]
    want = ref.rows_attention(f64(q), start, keys, values, seen, 0.1)
    check(out, lse, want, 100, D, "bad")
    assert not bool(out[start[5]:].any())  # no page of its own at all


def test_bad_row_starts(V):
    n, Hq, D = 60, 2, 64
    rng = np.random.default_rng(1)
    q, k, v = bf16(rng, (n, Hq, D)), bf16(rng, (n, 1, D)), bf16(rng, (n, 1, D))
    for start, zero, kept in (([-5, 10, 20], slice(0, 10), slice(20, n)), ([0, 10, n + 9], slice(10, n), slice(0, 0)),
                              ([30, 20, 40], slice(0, 0), slice(40, n))):
        out, lse, _ = buffers(n, Hq, D, False)
        ws = workspace(V.vp_prompt_attention_workspace_bytes(2, n, Hq, 1, D))
        V.vp_prompt_attention(q, Hq * D, k, D, v, D, i32(start), 2, n, Hq, 1, D, 0.1, None, out, lse, ws)
        torch.cuda.synchronize()
        assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
        assert not bool(out[zero].any()) and bool(torch.isneginf(lse[zero]).all()) and bool((out[kept] == 7.0).all())


# ------------------------------------------------------------------ workspaces, graphs, streams, large caches
def test_graph_replays_with_new_inputs_and_lengths(V):
    S, Hq, Hkv, D, P = 3, 24, 4, 256, 64
    c = Cache(V, 2, S, 40, P, Hkv, D, False)
    start, M = i32([0, 8, 16, 24]), 24
    q, L = bf16(np.random.default_rng(1), (M, Hq, D)), i32([100, 2000, 8])
    out = torch.empty_like(q)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    call = lambda: c.attend(q, start, L, M, Hq, D ** -0.5, None, out, None, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    q2, L2 = bf16(np.random.default_rng(2), (M, Hq, D)), [2500, 33, 64]
    want = torch.empty_like(q)
    c.attend(q2, start, i32(L2), M, Hq, D ** -0.5, None, want, None, workspace(ws.numel()))
    q.copy_(q2)
    L.copy_(i32(L2))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_streams_and_a_workspace_in_turn_with_the_other_served_calls(V):
    S, Hq, Hkv, D, P = 4, 8, 2, 128, 32
    cs = [Cache(V, i, S, 50, P, Hkv, D, i % 2 == 1) for i in range(4)]
    rows, L = [1, 7, 130, 2], [1500, 900, 130, 64]
    start = np.cumsum([0] + rows)
    M = int(start[-1])
    q = bf16(np.random.default_rng(1), (M, Hq, D))
    need = V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D)
    want = []
    for c in cs:
        out = torch.empty_like(q)
        c.attend(q, i32(start), i32(L), M, Hq, 0.1, None, out, None, workspace(need))
        want.append(out)
    torch.cuda.synchronize()
    sts, wss, outs = [torch.cuda.Stream() for _ in cs], [workspace(need) for _ in cs], [torch.empty_like(q) for _ in cs]
    st, ln = i32(start), i32(L)
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, w, o in zip(cs, sts, wss, outs):
            c.attend(q, st, ln, M, Hq, 0.1, None, o, None, w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    # one workspace: single tokens (whose counters lie in it), rows, prompts in turn
    ws = workspace(max(need, V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D), V.vp_prompt_attention_workspace_bytes(1, M, Hq, Hkv, D)))
    one, first = q[:S].contiguous(), None
    kv = bf16(np.random.default_rng(3), (M, 2 * Hkv, D))
    for _ in range(3):
        o1, o2, o3 = torch.empty_like(one), torch.empty_like(q), torch.empty_like(q)
        V.vp_paged_attention(cs[0].desc(), one, ln, S, Hq, 0.1, None, o1, None, ws)
        cs[0].attend(q, st, ln, M, Hq, 0.1, None, o2, None, ws)
        V.vp_prompt_attention(q, Hq * D, kv, 2 * Hkv * D, kv[:, Hkv:], 2 * Hkv * D, i32([0, M]), 1, M, Hq, Hkv, D, 0.1, None, o3, None, ws)
        first = first or (o1, o2, o3)
        assert torch.equal(o2, want[0]) and torch.equal(o1, first[0]) and torch.equal(o3, first[2])
    assert V.vp_read_status(ws) == V.VP_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_beyond_32_bits(V, fp8):
    D, Hkv, P = 256, 8, 128
    n_pages = (1 << 32) // (D * Hkv * P) + 40  # more than 2^32 elements
    try:
        dt = torch.uint8 if fp8 else torch.bfloat16
        k, v = (torch.zeros((n_pages, Hkv, P, D), dtype=dt, device="cuda") for _ in "kv")
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    c = Cache(V, 1, 1, 4, P, Hkv, D, fp8)
    ids = np.array([[n_pages - 1, 3, n_pages - 7, n_pages - 2]], np.int32)
    for i in range(4):
        k[int(ids[0, i])], v[int(ids[0, i])] = c.k[int(c.table[0, i])], c.v[int(c.table[0, i])]
    if fp8:
        ks, vs = (torch.zeros((n_pages, Hkv, P), dtype=torch.uint8, device="cuda") for _ in "kv")
        for i in range(4):
            ks[int(ids[0, i])], vs[int(ids[0, i])] = c.ks[int(c.table[0, i])], c.vs[int(c.table[0, i])]
    n, L, Hq = 5, 500, 16
    q = bf16(np.random.default_rng(1), (n, Hq, D))
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, n, Hq, Hkv, D))
    want, got = torch.empty_like(q), torch.empty_like(q)
    c.attend(q, i32([0, n]), i32([L]), n, Hq, 0.1, None, want, None, ws)
    pages = i32(ids)
    if fp8:
        V.vp_paged_attention_rows_fp8(V.vp_paged_cache_fp8(k, v, ks, vs, pages, n_pages, P, 4, Hkv, D), q, i32([0, n]), i32([L]), 1, n,
                                      Hq, 0.1, None, got, None, ws)
    else:
        V.vp_paged_attention_rows(V.vp_paged_cache(k, v, pages, n_pages, P, 4, Hkv, D), q, i32([0, n]), i32([L]), 1, n, Hq, 0.1, None,
                                  got, None, ws)
    assert torch.equal(want, got)


# ------------------------------------------------------------------ the 8-bit cache's append
def codes_equal(got, want):
    return np.array_equal(ref.e4m3_value(got), want)


@pytest.mark.parametrize("D,Hq,Hkv,P,rot,inter,norm", [
    (256, 24, 4, 64, 256, True, True), (256, 6, 1, 16, 64, False, True), (128, 32, 8, 16, 128, False, False),
    (128, 5, 5, 32, 96, False, True), (64, 8, 2, 128, 64, True, False), (64, 3, 1, 64, 16, False, True), (128, 4, 2, 64, 0, True, False),
    (256, 6, 2, 32, 64, False, False), (128, 4, 4, 16, 32, True, False), (64, 1, 3, 16, 16, False, False)])  # a part rotates, no norm
def test_append_fp8(V, D, Hq, Hkv, P, rot, inter, norm):
    rng = np.random.default_rng(D + rot)
    rows, ctx = [1, 0, P + 3, 2, 400], [0, 5, P - 2, 3 * P - 1, 2 * P]
    S, T = len(rows), sum(rows)
    start = np.cumsum([1] + rows)
    M = T + 2
    mp = -(-max(a + b for a, b in zip(rows, ctx)) // P)
    c, c16 = Cache(V, D + P, S, mp, P, Hkv, D, True), Cache(V, D + P, S, mp, P, Hkv, D, False)
    ld = (Hq + 2 * Hkv) * D + 24
    x = bf16(rng, (M, ld)) * torch.exp2(torch.randint(-20, 20, (M, 1), device="cuda").float()).to(torch.bfloat16)
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]
    k[2], v[3] = 0.0, 0.0
    qn = f32(rng.uniform(0.5, 1.5, D)) if norm else None
    kn = f32(rng.uniform(0.5, 1.5, D)) if norm else None
    rope = V.vp_rope(freqs(rot), inter) if rot else None
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    q_out, q16 = (torch.full((M, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kv_len, status = i32([-9] * S), i32([0])
    args = (q, ld, k, ld, v, ld, qn, kn, 1e-6, rope, i32(start), i32(ctx), S, M, Hq)
    V.vp_paged_append_fp8(c.desc(), *args, q_out, kv_len, status)
    V.vp_paged_append(c16.desc(), *args, q16)
    torch.cuda.synchronize()
    assert int(status) == 0 and kv_len.tolist() == [a + b for a, b in zip(ctx, rows)]
    assert torch.equal(q_out.view(torch.int16), q16.view(torch.int16))  # the queries, and padding rows
    seq = np.repeat(np.arange(S), rows)
    pos = np.concatenate([a + np.arange(n) for a, n in zip(ctx, rows)])
    at = torch.from_numpy(c.table[seq, pos // P]).cuda().long(), torch.from_numpy(pos % P).cuda()
    xk = f64(k[1:1 + T]).reshape(T, Hkv, D)
    want_k, _ = ref.norm_rope(xk, f64(kn) if norm else None, 1e-6, pos, freqs(rot) if rot else [], inter)
    for want, got, sc in ((want_k, c.k, c.ks), (f64(v[1:1 + T]).reshape(T, Hkv, D), c.v, c.vs)):
        y, e = ref.pow2_codes(want)
        assert np.array_equal(sc[at[0], :, at[1]].cpu().numpy().astype(int) - 127, e)
        assert codes_equal(got[at[0], :, at[1]].cpu().numpy(), y)
    for t, b in zip((c.k, c.v, c.ks, c.vs), before):  # nothing else changed
        t[at[0], :, at[1]] = b[at[0], :, at[1]]
        assert torch.equal(t, b)


def test_append_fp8_borders_ties_and_values_that_are_none(V):
    """Maxima at 448 2^e and next to it, values half way between codes, subnormal heads, infinities and NaN."""
    D, P, rows = 64, 16, 12
    c = Cache(V, 1, 1, 1, P, 1, D, True)
    x = np.zeros((rows, D))
    x[0, :4] = [448.0, 1.0625, 1.1875, -2.125]  # ties, to the even code
    x[1, :2] = [450.0, 1.0]                     # the next scale
    x[2, 0] = 2.0 ** -133                       # bf16's smallest
    x[3, :3] = [2.0 ** 127, -(2.0 ** 127) * 1.75, 1.0]
    x[4, :3] = [448.0, 2.0 ** -9 * 1.5, 2.0 ** -9 * 0.5]  # below e4m3's smallest normal: ties
    x[5, 0], x[6, 1] = np.inf, np.nan
    x[7] = -3.0
    x[8, :2] = [0.875 * 2.0 ** -100, 2.0 ** -110]
    x[9, :2] = [-0.8828125 * 2.0 ** 40, 2.0 ** 30]
    kv = torch.from_numpy(x).to(torch.bfloat16).cuda()
    V.vp_paged_append_fp8(c.desc(), None, 0, kv, D, kv, D, None, None, 0.0, None, i32([0, rows]), i32([0]), 1, rows, 0, None)
    xx = f64(kv)
    fin = np.isfinite(xx).all(1)
    y, e = ref.pow2_codes(xx[fin])
    for codes, sc in ((c.k, c.ks), (c.v, c.vs)):
        got, gs = codes[int(c.table[0, 0]), 0, :rows].cpu().numpy(), sc[int(c.table[0, 0]), 0, :rows].cpu().numpy()
        assert codes_equal(got[fin], y) and np.array_equal(gs[fin].astype(int) - 127, e)
        assert (gs[~fin] == 255).all() and (got[~fin] == 0x7F).all()


def test_append_fp8_keys_next_to_borders(V):
    """Normed keys whose exact values lie next to ties and whose maxima lie next to 448 2^e: the exact value's codes."""
    D, P, T = 128, 128, 2048
    c = Cache(V, 1, 1, T // P, P, 1, D, True)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randint(1, 9, (T, D), generator=g, device="cuda").to(torch.bfloat16)  # few mantissa bits: many products near ties
    w = f32(np.full(D, 1.0))
    V.vp_paged_append_fp8(c.desc(), None, 0, k, D, k, D, None, w, 1e-6, V.vp_rope([0.0] * (D // 2), False), i32([0, T]), i32([0]), 1, T,
                          0, None)
    want, _ = ref.norm_rope(f64(k).reshape(T, 1, D), np.ones(D), 1e-6, np.arange(T), [0.0] * (D // 2), False)
    y, e = ref.pow2_codes(want)
    pg = torch.from_numpy(c.table[0, np.arange(T) // P]).cuda().long(), torch.arange(T, device="cuda") % P
    assert np.array_equal(c.ks[pg[0], :, pg[1]].cpu().numpy().astype(int) - 127, e)
    assert codes_equal(c.k[pg[0], :, pg[1]].cpu().numpy(), y)


def test_append_fp8_bad_pages_and_positions(V):
    D, P, Hq, Hkv, S = 128, 16, 2, 1, 4
    c = Cache(V, 2, S, 2, P, Hkv, D, True)
    c.table[1, 0], c.table[2, 1] = -1, c.n
    c.pages = i32(c.table)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    x = bf16(np.random.default_rng(1), (S, Hq + 2 * Hkv, D))
    out, status = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda"), i32([0])
    ld = (Hq + 2 * Hkv) * D
    V.vp_paged_append_fp8(c.desc(), x, ld, x[:, Hq:], ld, x[:, Hq + Hkv:], ld, None, None, 0.0, None, None, i32([3, 3, 20, 32]), S, S, Hq, out,
                          None, status)
    assert int(status) == V.VP_ERR_SHAPE and not bool(out[1:].any()) and torch.equal(out[0], x[0, :Hq])
    pg = int(c.table[0, 0])
    for t, b in zip((c.k, c.v, c.ks, c.vs), before):
        assert not torch.equal(t[pg, :, 3], b[pg, :, 3])
        t[pg, :, 3] = b[pg, :, 3]
        assert torch.equal(t, b)


# ------------------------------------------------------------------ the calls together
def test_prompt_in_chunks_and_single_tokens_equal_the_whole_prompt(V):
    """A prompt through the bf16 cache in chunks and single tokens, as a server runs it, against one call of the whole prompt
    on the same keys; and the 8-bit cache against its own definition."""
    T, Hq, Hkv, D, P = 300, 24, 4, 256, 64
    rng = np.random.default_rng(5)
    x = bf16(rng, (T, Hq + 2 * Hkv, D))
    ld, w, rope = (Hq + 2 * Hkv) * D, f32(rng.uniform(0.5, 1.5, D)), V.vp_rope(freqs(D), True)
    c, c8 = Cache(V, 1, 1, 5, P, Hkv, D, False), Cache(V, 2, 1, 5, P, Hkv, D, True)
    outs, outs8, qs, at = [], [], [], 0
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, T, Hq, Hkv, D))
    for n in (130, 1, 8, 1, 100, 60):
        part, ctx, L = x[at:at + n], i32([at]), i32([0])
        for cache, app, res in ((c, V.vp_paged_append, outs), (c8, V.vp_paged_append_fp8, outs8)):
            q = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
            app(cache.desc(), part, ld, part[:, Hq:], ld, part[:, Hq + Hkv:], ld, w, w, 1e-6, rope, i32([0, n]), ctx, 1, n, Hq, q, L)
            o = torch.empty_like(q)
            cache.attend(q, i32([0, n]), L, n, Hq, D ** -0.5, None, o, None, ws)
            res.append(o)
        qs.append(q)
        at += n
    q = torch.cat(qs)
    k, v, _ = c.values(0, T)
    want, n = want_of(q, [0, T], [k], [v], [0], None, D ** -0.5, None)
    check(torch.cat(outs), None, want, n, D, "chunks")
    whole, kv = torch.empty_like(q), torch.from_numpy(np.stack([k, v], 1)).cuda().to(torch.bfloat16)
    V.vp_prompt_attention(q, Hq * D, kv, 2 * Hkv * D, kv[:, 1], 2 * Hkv * D, i32([0, T]), 1, T, Hq, Hkv, D, D ** -0.5, None, whole, None, ws)
    check(whole, None, want, n, D, "whole")
    k8, v8, _ = c8.values(0, T)
    want8, n = want_of(q, [0, T], [k8], [v8], [0], None, D ** -0.5, None)
    check(torch.cat(outs8), None, want8, n, D, "chunks in 8 bits")
    assert math.isfinite(float(torch.cat(outs8).float().abs().max()))
