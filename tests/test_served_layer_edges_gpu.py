"""GPU tests of the served attention layer's operators at their edges.  Tolerances as in test_served_layer_gpu.py,
unless a test derives its own."""
import numpy as np
import pytest
import torch

from helpers import workspace
from oracle import served_layer as ref
from test_served_layer_gpu import (U, Paged, assert_codes, assert_within, attend, bf16, f32, f64, freqs, i32, linear,
                                   nearest_codes, run_norm)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


# ------------------------------------------------------------------ status
def preset(ws, value):
    ws[:4].view(torch.int32).fill_(value)
    return ws


@pytest.mark.parametrize("before,after", [("VP_OK", "VP_ERR_SHAPE"), ("VP_ERR_TIMEOUT", "VP_ERR_TIMEOUT")])
def test_a_bad_length_or_page_does_not_hide_a_timeout(V, before, after):
    """A timed-out call leaves counters behind, so its report must stand until the workspace is zero-filled."""
    rng = np.random.default_rng(1)
    P, D = 32, 128
    p = Paged(V, 2, 3, 4, P, 2, D)
    q = bf16(rng, (3, 4, D), 1.5)
    n = V.vp_paged_attention_workspace_bytes(3, 4, 2, D)
    attend(V, p, q, [100, -1, 20], D ** -0.5, ws=preset(workspace(n), getattr(V, before)), expect=getattr(V, after))
    p.pages[2, 0] = p.n
    attend(V, p, q, [100, 0, 20], D ** -0.5, ws=preset(workspace(n), getattr(V, before)), expect=getattr(V, after))
    status = i32([getattr(V, before)])
    k, v = bf16(rng, (3, 2, D)), bf16(rng, (3, 2, D))
    for start in (None, i32([0, 1, 2, 9])):
        V.vp_paged_append(p.desc(), None, 0, k, 2 * D, v, 2 * D, None, None, 0.0, None, start, i32([1, 1, -1]), 3, 3, 0, None,
                          None, status)
        assert int(status) == getattr(V, after)


# ------------------------------------------------------------------ codes after the norm
def exact_codes(h, w, K):
    """Codes (without sign) of the exact quotients h w 448 / max of every group: the row's factor cancels; h w has 32
    bits and 448 h w 35, so that the fp64 division rounds once and meets every tie."""
    return nearest_codes(f64(h) * (1.0 if w is None else f64(w)), K)[0]


WEIGHTS = {"none": lambda rng, K: None, "ones": lambda rng, K: np.ones(K), "tenths": lambda rng, K: np.full(K, 0.1),
           "bf16": lambda rng, K: bf16(rng, K, 0.1).double().cpu().numpy() + 1.0, "random": lambda rng, K: rng.uniform(-2, 2, K)}


def weights(rng, K, kind):
    w = WEIGHTS[kind](rng, K)
    if w is None:
        return None
    return f32(w) if kind != "bf16" else torch.from_numpy(w).to(torch.bfloat16).float().cuda()


@pytest.mark.parametrize("M", [5, 700])
@pytest.mark.parametrize("kind", ["none", "ones", "tenths", "bf16", "random"])
@pytest.mark.parametrize("wide", [False, True])
def test_add_rmsnorm_codes_are_the_exact_quotients(V, M, kind, wide):
    """Every code, ties and the codes below e4m3's smallest normal value among them."""
    rng = np.random.default_rng(M)
    K = 2064
    x = rng.standard_normal((M, K)) * 2.0 ** -(rng.integers(0, 3, (M, K)) * rng.integers(0, 9, (M, K)))
    x = f32(x) if wide else f32(x).to(torch.bfloat16)
    w = weights(rng, K, kind)
    h, q, _ = run_norm(V, x, None, w, 1e-6, K)
    assert np.array_equal(q & 127, exact_codes(h, w, K))


@pytest.mark.parametrize("kind", ["none", "ones", "tenths"])
@pytest.mark.parametrize("rows", [1, 320])
def test_add_rmsnorm_codes_of_every_pair_of_eight_bits(V, kind, rows):
    """Group a: the largest value a, and 127 others over every power of two down to the smallest codes."""
    K = 128 * 128
    a, b, e = np.arange(128, 256)[:, None], np.arange(128, 255)[None, :], np.arange(0, 22)[:, None, None]
    x = np.concatenate([np.broadcast_to(a * 1.0, (22, 128, 1)), b * 2.0 ** -(e + 1) * (1 - 2 * (b % 2)) * np.ones((1, 128, 1))], axis=2)
    x = x.reshape(22, K)
    x = torch.from_numpy(np.tile(x, (max(1, rows // 22), 1))).to(torch.bfloat16).cuda()
    w = weights(None, K, kind)
    h, q, _ = run_norm(V, x, None, w, 1e-6, K)
    assert np.array_equal(q & 127, exact_codes(h, w, K))


# ------------------------------------------------------------------ outside fp32's range
@pytest.mark.parametrize("M", [5, 400])
@pytest.mark.parametrize("what", ["weights", "rows"])
@pytest.mark.parametrize("wide", [False, True])
def test_add_rmsnorm_codes_outside_the_range_of_fp32(V, M, what, wide):
    """Products of 2^-100 and of 2^110 (the row's factor is about 1), and rows whose squares fp32 does not hold (about
    1e-21 and 1e21): codes of the exact quotients there, too."""
    rng = np.random.default_rng(M)
    K = 1040
    x = rng.standard_normal((M, K)) * 2.0 ** -rng.integers(0, 16, (M, K))
    w = np.ones(K)
    if what == "weights":
        w[:384], w[384:768] = 2.0 ** -100, 2.0 ** 110
    else:
        x *= np.where(np.arange(M) % 2, 2.0 ** -70, 2.0 ** 70)[:, None]
        w[::3] = 1.0 + 2.0 ** -6
    x = f32(x) if wide else f32(x).to(torch.bfloat16)
    h, q, s = run_norm(V, x, None, f32(w), 1e-30, K)
    assert np.array_equal(q & 127, exact_codes(h, f32(w), K))
    _, y = ref.add_rmsnorm(f64(x), None, f64(f32(w)), 1e-30)
    assert_codes(q, s, y, 40 * U, what)


@pytest.mark.parametrize("M", [3, 400])
def test_add_rmsnorm_values_above_fp32_have_finite_scales(V, M):
    """y reaches sqrt(K) times the weight: beyond fp32, while max / 448 is not."""
    K = 4096
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    x[:, 5], x[:, 6], x[:, 200] = 3.0, -1.0, 1.0
    w = torch.full((K,), 3e38, device="cuda")
    _, q, s = run_norm(V, x, None, w, 1e-6, K)
    _, y = ref.add_rmsnorm(f64(x), None, f64(w), 1e-6)
    assert np.abs(y).max() > 1e40
    assert_codes(q, s, y, 40 * U, "above fp32")


# ------------------------------------------------------------------ the largest eps
@pytest.mark.parametrize("eps", [1e38, 3.4e38])
def test_norms_with_the_largest_eps(V, eps):
    """mean + eps leaves fp32, its root does not."""
    rng = np.random.default_rng(7)
    x = bf16(rng, (3, 16), 4e18)
    h, q, s = run_norm(V, x, None, None, eps, 16)
    _, y = ref.add_rmsnorm(f64(x), None, None, eps)
    assert np.abs(y).max() > 0.1
    assert_codes(q, s, y, 40 * U, "norm")
    D, P = 64, 16
    p = Paged(V, 8, 3, 1, P, 1, D)
    k, w = bf16(rng, (3, 1, D), 2e18), torch.ones(D, device="cuda")
    V.vp_paged_append(p.desc(), None, 0, k, D, k, D, None, w, eps, None, None, i32([0, 0, 0]), 3, 3, 0, None)
    want, mag = ref.norm_rope(f64(k), np.ones(D), eps, np.zeros(3), [], False)
    assert np.abs(want).max() > 0.1
    assert_within(f64(p.k[p.pages[:, 0].long(), :, 0]), want, 2.0 ** -8 * np.abs(want) + 32 * U * mag, "append")


# ------------------------------------------------------------------ attention: gates
def test_attention_gates_near_the_end_of_the_exponents(V):
    """sigmoid of -80 and below times values up to bf16's largest: a product that bf16 holds is not lost."""
    S, Hq, Hkv, D, P = 2, 4, 2, 64, 16
    rng = np.random.default_rng(3)
    p = Paged(V, 4, S, 2, P, Hkv, D)
    p.v[:] = torch.from_numpy(rng.choice([-1.0, 1.0], p.v.shape) * 2.0 ** rng.choice([0, 3, 60, 120], p.v.shape[:3])[..., None]).to(
        torch.bfloat16).cuda()
    q = bf16(rng, (S, Hq, D))
    gate = torch.from_numpy(rng.uniform(-175, -80, (S, Hq, D))).to(torch.bfloat16).cuda()
    gate[0, :, :4] = torch.tensor([0.0, 30.0, 200.0, -50.0], dtype=torch.bfloat16)
    gate[1, 0, :2] = torch.tensor([float("-inf"), float("inf")], dtype=torch.bfloat16)
    lens = [1, 1]  # one key: the output is its value times the gate's sigmoid
    out, _ = attend(V, p, q, lens, D ** -0.5, gate)
    want, mag, _, _ = ref.paged_attention(f64(q), f64(p.k), f64(p.v), p.table, lens, D ** -0.5, f64(gate))
    assert (np.abs(want) > 1e-3).any() and ((np.abs(want) < 1e-37) & (np.abs(want) > 1e-40)).any()
    # an exponential of half the gate, 2 ulp, used twice, three products: below 2^-19; bf16's half step, 2^-134 below its normal values
    assert_within(f64(out), want, 2.0 ** -19 * mag + np.maximum(2.0 ** -8 * np.abs(want), 2.0 ** -134), "gate")


# ------------------------------------------------------------------ kernels of large calls
def append_cases():  # (D, Hq, Hkv, norm)
    for D in (64, 128, 256):
        for per in range(1, 7):
            for norm in (False, True):
                yield D, 128 * 8 // D * per - 3, 1, norm
    yield 256, 20, 4, True    # seven turns: two blocks a row
    yield 128, 32, 8, True
    yield 64, 96, 24, False


@pytest.mark.parametrize("D,Hq,Hkv,norm", list(append_cases()))
def test_append_of_many_rows(V, D, Hq, Hkv, norm):
    """Prompts: several heads per group of lanes (one to six), ragged sequences, padding rows at both ends."""
    rng = np.random.default_rng(D + Hq)
    P, inter = (16, True) if Hq % 2 else (64, False)
    rot = D if norm else D // 2
    at_once = 1024 // D
    turns = -(-(Hq + 2 * Hkv) // at_once)
    T = 16 * 160 // turns + 7  # 16 rows per SM and turn: past the rule for many
    cut = np.sort(rng.integers(0, T + 1, 3))
    rows = np.diff(np.concatenate([[0], cut, [T]]))
    rows = np.concatenate([rows[:2], [0], rows[2:]])
    S, ctx = len(rows), np.array([0, P - 1, 3, 2 * P, 5])
    M = T + 3
    max_pages = int(-(-(ctx + rows).max() // P)) + 1
    p = Paged(V, D + Hq, S, max_pages, P, Hkv, D)
    ld = (Hq + 2 * Hkv) * D + 8
    x = bf16(rng, (M, ld))
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]
    qn, kn = (f32(rng.uniform(0.5, 1.5, D)) for _ in range(2)) if norm else (None, None)
    want_k, want_v = p.k.clone(), p.v.clone()
    q_out = torch.full((M, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kv_len, status = i32([-9] * S), i32([0])
    start = 2 + np.concatenate([[0], np.cumsum(rows)])
    V.vp_paged_append(p.desc(), q, ld, k, ld, v, ld, qn, kn, 1e-6, V.vp_rope(freqs(rot), inter), i32(start), i32(ctx), S, M, Hq,
                      q_out, kv_len, status)
    torch.cuda.synchronize()
    assert int(status) == 0 and kv_len.tolist() == (ctx + rows).tolist()
    assert bool((q_out[:2] == 7.0).all()) and bool((q_out[2 + T:] == 7.0).all())
    seq = np.repeat(np.arange(S), rows)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, rows)])
    pg, sl = torch.from_numpy(p.table[seq, pos // P]).cuda().long(), torch.from_numpy(pos % P).cuda()
    got_k = p.k[pg, :, sl]
    for name, src, w, H, got in (("q", q, qn, Hq, q_out[2:2 + T]), ("k", k, kn, Hkv, got_k)):
        xin = f64(src[2:2 + T]).reshape(T, H, D)
        want, mag = ref.norm_rope(xin, f64(w) if norm else None, 1e-6, pos, freqs(rot), inter)
        assert_within(f64(got), want, 2.0 ** -8 * np.abs(want) + 32 * U * mag, f"append {name}")
        if not norm:
            assert np.array_equal(f64(got)[..., rot:], xin[..., rot:])
    want_k[pg, :, sl], want_v[pg, :, sl] = got_k, v[2:2 + T].reshape(T, Hkv, D)
    assert torch.equal(p.k, want_k) and torch.equal(p.v, want_v)  # the rows' slots alone have changed


def linear_plain(xq, xs, wq, ws):
    """The definition in fp64 on the device, 4,096 weight rows at a time -> (y, sum |x w|)."""
    K = xq.shape[1]
    spread = lambda s: s.double().repeat_interleave(128, 1)[:, :K]  # noqa: E731
    x = xq.view(torch.float8_e4m3fn).double() * spread(xs)
    ys, mags = [], []
    for n in range(0, wq.shape[0], 4096):
        w = wq[n:n + 4096]
        w = w.view(torch.float8_e4m3fn).double() * spread(ws[n // 128:(n + 4096) // 128].repeat_interleave(128, 0)[:len(w)])
        ys.append(x @ w.t())
        mags.append(x.abs() @ w.abs().t())
    return torch.cat(ys, 1), torch.cat(mags, 1)


@pytest.mark.parametrize("M,N,K", [(8, 19600, 5136), (24, 19600, 5136), (60, 19600, 5136), (100, 19600, 5136),
                                   (16, 39040, 2064), (32, 39040, 2064), (64, 39040, 2064), (128, 39040, 2064),
                                   (1024, 5120, 5120), (1000, 5136, 5136), (300, 20496, 528)])
def test_linear_block_of_more_tiles_than_ctas(V, M, N, K):
    """Whole rounds of output tiles, then a remainder: cut along K (and joined) for the longer K."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    code = lambda *s: torch.randint(0, 255, s, generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    xq, wq = code(M, K), code(N, K)
    for t in (xq, wq):
        t[(t & 127) == 127] = 0x30
    kb, nb = -(-K // 128), -(-N // 128)
    xs = (0.5 + torch.rand((M, kb), generator=g, device="cuda")) * 1e-2
    ws = (0.5 + torch.rand((nb, kb), generator=g, device="cuda")) * 1e-3
    want, mag = linear_plain(xq, xs, wq, ws)
    bound = 2 * (130 + kb) * U * mag + 1e-30
    wsp = workspace(V.vp_linear_fp8_block_workspace_bytes(M, N, K))
    y32 = linear(V, xq, xs, wq, ws, True, wsp=wsp)
    assert bool(((y32.double() - want).abs() <= bound).all())
    y16 = linear(V, xq, xs, wq, ws, False, wsp=wsp)
    assert bool(((y16.double() - want).abs() <= bound + 2.0 ** -8 * want.abs()).all())
    assert torch.equal(linear(V, xq, xs, wq, ws, True, wsp=wsp), y32)
