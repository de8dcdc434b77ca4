"""GPU tests of the attention of several new rows and of the 8-bit cache at their edges.  Tolerances as in
test_rows_attention_gpu.py, unless a test derives its own."""
import numpy as np
import pytest
import torch

from helpers import workspace
from oracle import served_layer as ref  # noqa: F401
from test_rows_attention_gpu import Cache, buffers, check, want_of
from test_served_layer_gpu import bf16, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


# ------------------------------------------------------------------ few rows: warps some of whose lanes have nothing to write
@pytest.mark.parametrize("D,G,n", [(64, 1, 1), (64, 4, 1), (128, 4, 1), (256, 4, 1), (256, 3, 1), (128, 9, 1), (64, 5, 5), (128, 31, 1),
                                   (256, 6, 5), (128, 1, 13), (256, 32, 1)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_rows_that_fill_a_warp_in_part(V, D, G, n, fp8, gate):
    """1 to 32 rows per key head: a warp writes eight of them, four lanes each, and the others of its lanes nothing."""
    S, P, Hkv, L = 5, 32, 2, [n + 70, n, n + 600, n + 128, 2500]
    c, M, Hq = Cache(V, D + G, S, -(-2500 // P), P, Hkv, D, fp8), S * n, G * Hkv
    q, start = bf16(np.random.default_rng(G), (M, Hq, D), 1.5), np.arange(S + 1) * n
    out, lse, g = buffers(M, Hq, D, gate)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(start), i32(L), M, Hq, D ** -0.5, g, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    kv = [c.values(s, L[s]) for s in range(S)]
    want, m = want_of(q, start, [x[0] for x in kv], [x[1] for x in kv], [a - n for a in L], None, D ** -0.5, g)
    check(out, lse, want, m, D, f"{D} {G} {n}")
    # one row at a time, whatever lies beside it in the warp: the same keys in the same order, but for where the work is cut
    one = torch.empty_like(out)
    for i in range(n):
        part = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda")
        rows = torch.arange(S, device="cuda") * n + i
        c.attend(q[rows].contiguous(), None, i32([a - n + i + 1 for a in L]), S, Hq, D ** -0.5, None if g is None else g[rows].contiguous(),
                 part, None, ws)
        one[rows] = part
    check(one, None, want, m, D, f"one by one {D} {G} {n}")


# ------------------------------------------------------------------ missing pages
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,G,n,P", [(256, 6, 60, 16), (256, 4, 150, 128), (256, 2, 260, 64), (128, 8, 40, 32), (64, 3, 100, 16), (256, 4, 3, 16)])
def test_missing_pages_block_by_block(V, D, G, n, P, fp8):
    """Pages that are missing here and there among 50 blocks of keys, so that every note of them is used again for a block with
    other ones: in CTA pairs (256 columns, more than 128 rows), single CTAs, and with few rows."""
    Hkv, S, L = 1, 2, [n + 6000, n + 3210]
    c = Cache(V, D + P, S, -(-max(L) // P), P, Hkv, D, fp8)
    rng = np.random.default_rng(P)
    gone = rng.random(c.table.shape) < 0.3
    c.table[gone] = rng.choice([-1, c.n, c.n + 77, 2 ** 31 - 1, -2 ** 31], gone.sum())
    c.pages = i32(c.table)
    M, Hq, start = S * n, G * Hkv, np.arange(S + 1) * n
    q = bf16(rng, (M, Hq, D), 1.5)
    out, lse, _ = buffers(M, Hq, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(start), i32(L), M, Hq, D ** -0.5, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
    kv = [c.values(s, L[s]) for s in range(S)]
    want, m = want_of(q, start, [x[0] for x in kv], [x[1] for x in kv], [a - n for a in L], [x[2] for x in kv], D ** -0.5, None)
    check(out, lse, want, m, D, f"missing {D} {fp8}")


# ------------------------------------------------------------------ the longest sequences
def longest(V, D, G, n, P, fp8):
    """Just below 2^31 positions, nearly all of them the same few pages over and over, with scores 64 below those of the last
    positions (less what the other columns add: 5 sigma of 4 at most): together below 2^31 e^-40 = 1e-8 of the weight, 2^-26."""
    mp, low, hi = (2 ** 31 - 1) // P, 37, 640 // P
    L = mp * P
    c = Cache(V, 4, 1, 1, P, 1, D, fp8, spare=low + hi - 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((low + hi, 1, P, D), generator=g, device="cuda") for _ in "kv")
    k[..., 0] = 0.0
    k[:low, ..., 0] = -8.0
    if fp8:
        c.k, c.v = (x.mul(32.0).to(torch.float8_e4m3fn).view(torch.uint8) for x in (k, v))
        c.ks, c.vs = (torch.full((low + hi, 1, P), 122, dtype=torch.uint8, device="cuda") for _ in "kv")
    else:
        c.k, c.v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    c.n, c.max_pages = low + hi, mp
    c.pages = torch.randint(0, low, (mp,), generator=g, device="cuda", dtype=torch.int32)
    c.pages[mp - hi:] = torch.arange(low, low + hi, device="cuda", dtype=torch.int32)
    q = (0.25 * torch.randn((n, G, D), generator=g, device="cuda")).to(torch.bfloat16)
    q[..., 0] = 8.0
    out, lse, _ = buffers(n, G, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, n, G, 1, D))
    c.attend(q, i32([0, n]), i32([L]), n, G, 1.0, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    tail = hi * P  # the positions on pages of their own
    c.table = c.pages[mp - hi:].cpu().numpy().reshape(1, -1)
    kk, vv, _ = c.values(0, tail)
    want, m = want_of(q, [0, n], [kk], [vv], [tail - n], None, 1.0, None)
    check(out, lse, want, m, D, f"longest {D} {G}")


@pytest.mark.parametrize("D,G,n,fp8", [(256, 64, 3, False), (256, 64, 3, True), (128, 64, 3, False), (64, 30, 4, True), (128, 8, 1, False)])
def test_items_that_take_long(V, D, G, n, fp8):
    """Warps that have nothing to do in an item wait for as long as it takes the others: 0.3 s for 192 rows here."""
    longest(V, D, G, n, 128, fp8)


@pytest.mark.parametrize("D,G,n,P,fp8", [(64, 1, 1, 16, False), (64, 64, 3, 16, True), (128, 8, 1, 32, True), (256, 64, 3, 64, False),
                                         (256, 64, 3, 16, True), (64, 40, 13, 64, False)])
def test_lengths_whose_last_block_ends_beyond_2_31(V, D, G, n, P, fp8):
    """Pages shorter than a block: up to 2^31 - 16 positions, so that the length rounded up to blocks has 32 bits; 13 rows of 40
    heads are three items."""
    longest(V, D, G, n, P, fp8)


# ------------------------------------------------------------------ sequences that see nothing
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,G,rows", [(64, 2, [1, 2, 1]), (128, 8, [40, 3, 60]), (256, 4, [1, 1, 1]), (256, 6, [50, 30, 200])])
def test_zeros_of_bad_sequences_whatever_the_gate_holds(V, D, G, rows, fp8):
    c = Cache(V, 1, 3, 8, 64, 1, D, fp8)
    start = np.cumsum([0] + rows)
    M = int(start[-1])
    q = bf16(np.random.default_rng(1), (M, G, D))
    out, lse, g = buffers(M, G, D, True)
    g[start[1]:start[2]] = float("nan")
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(3, M, G, 1, D))
    L = [300, 513, 400]  # the second is behind its table
    c.attend(q, i32(start), i32(L), M, G, 0.1, g, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
    bad = slice(start[1], start[2])
    assert not bool(out[bad].any()) and bool(torch.isneginf(lse[bad]).all())
    kv = [c.values(s, 0 if s == 1 else L[s]) for s in range(3)]
    g[bad] = 0.0
    want, m = want_of(q, start, [x[0] for x in kv], [x[1] for x in kv], [L[s] - rows[s] for s in range(3)], None, 0.1, g)
    check(out, lse, want, m, D, "beside a bad one")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,G,lens", [(64, 2, [0, 100, 0, 1, 3000, 0]), (128, 4, [0] * 40), (256, 4, [7, 0, 0, 2000]),
                                      (128, 64, [0, 0, 65]), (256, 64, [0] * 3), (64, 1, [0] * 700 + [50] + [0] * 900)])
def test_empty_slots_are_no_error(V, D, G, lens, fp8):
    """Single tokens of a batch with idle slots, as the call for single tokens alone takes them: kv_len 0 gives zeros, lse -inf
    and VP_OK."""
    S, P = len(lens), 64
    c = Cache(V, 1, 1, 64, P, 1, D, fp8)
    c.S, c.max_pages, n = S, 64, max(max(lens), 1)
    c.table = np.repeat(c.table, S, 0)  # the same pages for all
    c.pages = i32(c.table)
    q = bf16(np.random.default_rng(1), (S, G, D), 1.5)
    out, lse, g = buffers(S, G, D, True)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, S, G, 1, D))
    c.attend(q, None, i32(lens), S, G, D ** -0.5, g, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    idle = torch.tensor([x == 0 for x in lens], device="cuda")
    assert not bool(out[idle].any()) and bool(torch.isneginf(lse[idle]).all())
    kv = [c.values(s, lens[s]) for s in range(S)]
    want, m = want_of(q, np.arange(S + 1), [x[0] for x in kv], [x[1] for x in kv], [x - 1 for x in lens], None, D ** -0.5, g)
    check(out, lse, want, m, D, f"idle {D}")
    # with row_start the same lengths do not fit, and a negative one never does
    for start, ls in ((np.arange(S + 1), lens), (None, [-1] + lens[1:])):
        c.attend(q, None if start is None else i32(start), i32(ls), S, G, D ** -0.5, g, out, lse, ws)
        torch.cuda.synchronize()
        assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
        V.vp_workspace_init(ws)
    check(out[1:], lse[1:], [w[1:] for w in want], m, D, f"negative {D}")


@pytest.mark.parametrize("source", ["prompt", "rows", "rows8"])
@pytest.mark.parametrize("start", [[0, 60, 0, 60, 0, 60], [5, 4], [0, 20, 40, 39, 60], list(range(50)) + [48, 60], [0, 2 ** 31 - 1, 0, 60],
                                   [30, -2 ** 31, 60], [0] * 1000 + [60] + [59] * 900 + [60]])
def test_a_row_start_that_decreases_writes_no_row(V, source, start):
    """Overlapping sequences would multiply the work without limit, and write the same rows twice."""
    D, Hq, Hkv, n, S = 128, 4, 2, 60, len(start) - 1
    rng = np.random.default_rng(1)
    q, k, v = bf16(rng, (n, Hq, D)), bf16(rng, (n, Hkv, D)), bf16(rng, (n, Hkv, D))
    out, lse, _ = buffers(n, Hq, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, n, Hq, Hkv, D))
    if source == "prompt":
        V.vp_prompt_attention(q, Hq * D, k, Hkv * D, v, Hkv * D, i32(start), S, n, Hq, Hkv, D, 0.1, None, out, lse, ws)
    else:
        c = Cache(V, 1, 1, 10, 16, Hkv, D, source == "rows8")
        c.S, c.pages = S, i32(np.repeat(c.table, S, 0))
        c.attend(q, i32(start), i32([100] * S), n, Hq, 0.1, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_ERR_SHAPE
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


# ------------------------------------------------------------------ scores beyond fp32's range
@pytest.mark.parametrize("D,G,n,long", [(64, 1, 1, 0), (128, 4, 2, 0), (128, 8, 90, 0), (256, 4, 70, 0), (256, 1, 3, 1), (128, 64, 5, 1)])
@pytest.mark.parametrize("fp8", [False, True])
def test_scores_beyond_the_range_are_no_zeros(V, D, G, n, long, fp8):
    """One key with a score of 2^130 makes the rows that see it NaN, one with -2^130 has no weight, and so do all of a row."""
    P, L = 64, 200 + 30_000 * long
    c = Cache(V, 1, 1, -(-L // P), P, 1, D, fp8)
    q = bf16(np.random.default_rng(1), (n, G, D))
    q[..., 0] = 2.0 ** 60
    pg = lambda t: (int(c.table[0, t // P]), 0, t % P)  # noqa: E731
    if fp8:
        c.k[..., 0] = 0  # no part in the other scores
    else:
        c.k[..., 0] = 0.0
    t = L - n + n // 2  # the rows from n // 2 on see it

    def put(t, sign):  # a key of 2^62 sign, alone in its column
        if fp8:
            c.k[pg(t)] = 0
            c.k[pg(t)][0] = 0x38 | (0x80 if sign < 0 else 0)
            c.ks[pg(t)] = 127 + 62
        else:
            c.k[pg(t)] = 0.0
            c.k[pg(t)][0] = sign * 2.0 ** 62

    def run():
        out, lse, _ = buffers(n, G, D, False)
        ws = workspace(V.vp_paged_attention_rows_workspace_bytes(1, n, G, 1, D))
        c.attend(q, i32([0, n]), i32([L]), n, G, 2.0 ** 8, None, out, lse, ws)
        torch.cuda.synchronize()
        assert V.vp_read_status(ws) == V.VP_OK
        return out, lse

    good, l0 = run()
    put(t, 1)
    out, lse = run()
    assert torch.equal(out[:n // 2], good[:n // 2]) and torch.equal(lse[:n // 2], l0[:n // 2])
    assert bool(torch.isnan(out[n // 2:]).all()) and bool(torch.isnan(lse[n // 2:]).all())
    put(t, -1)
    out, lse = run()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    c.k.zero_()
    c.k[..., 0] = 0xB8 if fp8 else -2.0 ** 62
    if fp8:
        c.ks.fill_(127 + 62)
    out, lse = run()
    assert not bool(out.any()) and bool(torch.isneginf(lse).all())


# ------------------------------------------------------------------ scale bytes behind the end
@pytest.mark.parametrize("D,G,n,L", [(128, 4, 1, 130), (256, 6, 1, 65), (64, 2, 3, 300), (128, 8, 40, 1000), (256, 4, 60, 201), (256, 4, 60, 190)])
def test_scale_bytes_behind_the_end_have_no_effect(V, D, G, n, L):
    """Any byte may lie there; large ones before the end are scales like others, beside whatever lies behind it."""
    S, P, M = 3, 128, 3 * n
    c = Cache(V, D, S, -(-L // P), P, 2, D, True)
    for s in range(S):
        c.vs[int(c.table[s, 0]), :, 3::7] = 140 + s
    q = bf16(np.random.default_rng(1), (M, 2 * G, D), 1.5)
    ws, outs = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, 2 * G, 2, D)), []
    for byte in (120, 0, 134, 135, 254, 255):
        for t in (c.ks, c.vs):
            for s in range(S):
                if L % P:
                    t[int(c.table[s, (L - 1) // P]), :, L % P:] = byte
        out, lse, _ = buffers(M, 2 * G, D, False)
        c.attend(q, i32(np.arange(S + 1) * n), i32([L] * S), M, 2 * G, D ** -0.5, None, out, lse, ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs)
    kv = [c.values(s, L) for s in range(S)]
    want, m = want_of(q, np.arange(S + 1) * n, [x[0] for x in kv], [x[1] for x in kv], [L - n] * S, None, D ** -0.5, None)
    check(out, lse, want, m, D, "scales behind the end")


def test_scale_bytes_behind_the_end_cost_nothing(V):
    """64 single tokens of 130 positions, 126 unused slots each: 41 us whatever lies there (77 where every large byte made its tile
    go the slow way).  The best of 20 runs; half as much again is allowed."""
    S, L, P, Hkv, D, Hq = 64, 130, 128, 8, 128, 32
    c = Cache(V, 1, S, 2, P, Hkv, D, True)
    q, ln = bf16(np.random.default_rng(1), (S, Hq, D)), i32([L] * S)
    out, ws, best = torch.empty_like(q), workspace(V.vp_paged_attention_rows_workspace_bytes(S, S, Hq, Hkv, D)), []
    for byte in (120, 255):
        for t in (c.ks, c.vs):
            t[torch.from_numpy(c.table[:, 1]).cuda().long(), :, L % P:] = byte
        times = []
        for _ in range(20):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in "ab")
            a.record()
            for _ in range(5):
                c.attend(q, None, ln, S, Hq, 0.1, None, out, None, ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        best.append(min(times))
    assert best[1] < 1.5 * best[0], best
