"""GPU parity of the served attention layer's operators (vp_quant_fp8, vp_add_rmsnorm_fp8,
vp_linear_fp8_block, vp_paged_append, vp_paged_attention) against the fp64 definitions in
oracle/served_layer.py, through the C ABI.

Tolerances, with u = 2^-24 (half an fp32 step) and the output's half step (bf16 2^-8; e4m3 2^-4, or
2^-10 below its smallest normal):
  scales     one rounding of max / 448 for the quantiser: 2 u; after the norm also the norm's own error.
  norm       sum of squares: at most 16 + 5 + 32 additions in a chain, halved by the root, plus the root,
             two divisions and two products: below 40 u.
  codes      x * (1 / s): 3 u more before the e4m3 rounding.
  linear     128 products exact in fp32, 128 additions inside a block and one per block outside, each
             at most 2 u (the tensor core may cut instead of rounding), two products: 2 (130 + KB) u of
             sum |x w|, then the output's half step.
  rope       norm as above with 8 + 5 additions (20 u), the angle as an fp32 fraction of a half turn (pi u / 2),
             sine and cosine (2 u each), two products: below 32 u of the pair's length.
  attention  a score's D products: 2 D u of scale * sum |q k| =: e (the same for the exponents' common factor log2 e,
             u of the score, itself below sum |q k|), weights exp(2 e) - 1 plus 2^-16 (the split of P, exp2, sums
             of up to n weights at u each), times sum p |v|; gate and division 8 u; then bf16's half step."""
import numpy as np
import pytest
import torch

import oracle
from helpers import workspace
from oracle import served_layer as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


def bits16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.double().cpu().numpy()


def bf16(rng, shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16).cuda()


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def assert_within(got, want, bound, what):
    err = np.abs(got - want)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside; first {i}: got {got[i]!r} want {want[i]!r} "
                             f"bound {bound[i]!r}")


def assert_codes(q, s, y, rel, what):
    """Device codes q and scales s of the exact values y, whose device forms are off by at most rel."""
    K = y.shape[1]
    want_s = ref.block_scales(y)
    assert_within(s, want_s, (rel + 2 * U) * want_s, what + " scales")
    t = y / ref.spread(s, K)
    half = np.maximum(2.0 ** -4 * np.abs(t), 2.0 ** -10)
    assert_within(ref.e4m3_value(q), t, half + (rel + 3 * U) * np.abs(t), what + " codes")


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (1, 128, 8), (3, 272, 0), (7, 144, 24), (130, 5120, 0), (2, 17408, 16),
                                     (1, 65536, 0)])
@pytest.mark.parametrize("wide", [False, True])
def test_quant(V, M, K, pad, wide):
    rng = np.random.default_rng(M + K)
    x = bf16(rng, (M, K + pad), 3.0)
    if wide:
        x = f32(rng.standard_normal((M, K + pad)) * 3.0)
    x[0, :16] = 0.0
    if K > 128:
        x[0, :128] = 0.0  # a whole group of zeros
        x[-1, 128:min(K, 256)] *= 1e-37  # scales near the smallest
    q = torch.full((M + 1, K), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((M + 1, -(-K // 128)), 7.0, device="cuda")
    V.vp_quant_fp8(x, V.VP_F32 if wide else V.VP_BF16, K + pad, M, K, q, s)
    torch.cuda.synchronize()
    assert_codes(q[:M].cpu().numpy(), f64(s[:M]), f64(x[:, :K]), 0.0, f"quant {M}x{K}")
    assert bool((q[M] == 0x5A).all()) and bool((s[M] == 7.0).all())  # nothing behind the last row


def test_quant_infinities_and_nan_reach_their_group_only(V):
    x = torch.ones((2, 400), dtype=torch.bfloat16, device="cuda")
    x[0, 130], x[1, 390] = float("nan"), float("-inf")
    q = torch.empty((2, 400), dtype=torch.uint8, device="cuda")
    s = torch.empty((2, 4), device="cuda")
    V.vp_quant_fp8(x, V.VP_BF16, 400, 2, 400, q, s)
    v, s = ref.e4m3_value(q.cpu().numpy()), s.cpu().numpy()
    assert np.isnan(s[0, 1]) and np.isinf(s[1, 3]) and np.isfinite(np.delete(s.ravel(), [1, 7])).all()
    assert np.isnan(v[0, 128:256]).all() and np.isnan(v[1, 390]) and not v[1, 384:390].any()
    assert np.all(v[0, :128] == 448) and np.all(v[0, 256:] == 448) and np.all(v[1, :384] == 448)


# ------------------------------------------------------------------ add + RMSNorm
def run_norm(V, x, residual, weight, eps, K, h="new"):
    M = x.shape[0]
    wide = x.dtype == torch.float32
    h = torch.empty((M, K), dtype=torch.bfloat16, device="cuda") if h == "new" else h
    q = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, -(-K // 128)), device="cuda")
    V.vp_add_rmsnorm_fp8(x, V.VP_F32 if wide else V.VP_BF16, x.stride(0), residual, weight, eps, M, K, h, q, s)
    torch.cuda.synchronize()
    return h, q.cpu().numpy(), f64(s)


@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (5, 5120, 0), (3, 16384, 0), (2, 8208, 16), (9, 272, 8), (4, 1152, 0),
                                     (1, 4096, 0)])
@pytest.mark.parametrize("wide,res,weight", [(False, True, True), (True, True, False), (False, False, True), (True, False, False)])
def test_add_rmsnorm(V, M, K, pad, wide, res, weight):
    rng = np.random.default_rng(M * K)
    x = f32(rng.standard_normal((M, K + pad))) if wide else bf16(rng, (M, K + pad))
    r = bf16(rng, (M, K), 4.0) if res else None
    w = f32(rng.uniform(-2, 2, K)) if weight else None
    x[0, 1] = 30.0
    h, q, s = run_norm(V, x, r, w, 1e-6, K)
    want_h, y = ref.add_rmsnorm(f64(x[:, :K]), bits16(r) if res else None, f64(w) if weight else None, 1e-6)
    assert np.array_equal(bits16(h), want_h)
    assert_codes(q, s, y, 40 * U, f"norm {M}x{K}")


def test_add_rmsnorm_in_place_and_without_h(V):
    rng = np.random.default_rng(3)
    x, r = bf16(rng, (6, 1040)), bf16(rng, (6, 1040))
    h, q, s = run_norm(V, x, r, None, 1e-5, 1040)
    r2 = r.clone()
    h2, q2, s2 = run_norm(V, x, r2, None, 1e-5, 1040, h=r2)
    assert torch.equal(h, r2) and np.array_equal(q, q2) and np.array_equal(s, s2)
    x2 = x.clone()
    _, q3, s3 = run_norm(V, x2, r, None, 1e-5, 1040, h=x2)
    assert torch.equal(h, x2) and np.array_equal(q, q3) and np.array_equal(s, s3)
    _, q4, s4 = run_norm(V, x, r, None, 1e-5, 1040, h=None)
    assert np.array_equal(q, q4) and np.array_equal(s, s4)


def test_add_rmsnorm_range(V):
    """Rows whose squares leave fp32's range, a zero row, an infinity, a NaN."""
    rng = np.random.default_rng(4)
    base = rng.standard_normal((7, 384))
    scale = np.array([1e30, 1e-25, 1e-38, 0.0, 1e19, 1.0, 1.0])[:, None]
    x = torch.from_numpy(base * scale).to(torch.bfloat16).cuda()
    x[5, 200], x[6, 10] = float("inf"), float("nan")
    h, q, s = run_norm(V, x, None, None, 1e-30, 384)
    want_h, y = ref.add_rmsnorm(f64(x), None, None, 1e-30)
    assert np.array_equal(bits16(h)[:5], want_h[:5])
    assert_codes(q[:5], s[:5], y[:5], 40 * U, "norm range")
    v = ref.e4m3_value(q)
    assert np.isnan(v[5, 200]) and not v[5, :128].any() and np.isnan(s[5, 1]) and np.isfinite(s[5, 0])
    assert np.isnan(v[6]).all() and np.isnan(s[6]).all()


E4M3 = ref.e4m3_value(np.arange(127))  # rising


def nearest_codes(y, K):
    """e4m3 magnitudes (codes without sign) of y * 448 / max of every group, one rounding, ties to even; and how far
    each is from the border between two codes, relative to it."""
    t = np.abs(y)
    for b in range(0, K, 128):
        t[:, b:b + 128] = t[:, b:b + 128] * 448.0 / t[:, b:b + 128].max(axis=1, keepdims=True)
    hi = np.clip(np.searchsorted(E4M3, t), 1, 126)
    border = (E4M3[hi - 1] + E4M3[hi]) / 2
    up = np.where(t == border, hi % 2 == 0, t > border)
    return (hi - 1 + up).astype(np.uint8), np.abs(t / border - 1), border


@pytest.mark.parametrize("M,K", [(3, 1040), (700, 1408)])
def test_quant_of_bf16_rounds_once(V, M, K):
    """Products of eight bits hit e4m3's ties; the fp64 quotient is exact there."""
    rng = np.random.default_rng(M)
    x = bf16(rng, (M, K))
    q = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, -(-K // 128)), dtype=torch.float32, device="cuda")
    V.vp_quant_fp8(x, V.VP_BF16, K, M, K, q, s)
    want, _, border = nearest_codes(f64(x), K)
    got = q.cpu().numpy() & 127
    normal = border > 2.0 ** -6  # below, a tie is met in no more than 24 bits of the product
    assert np.array_equal(got[normal], want[normal])
    assert np.abs(got.astype(int) - want).max() <= 1


@pytest.mark.parametrize("M,K,pad", [(700, 16384, 0), (1300, 8208, 8)])
@pytest.mark.parametrize("wide", [False, True])
def test_quant_of_many_groups(V, M, K, pad, wide):
    """Enough groups for several per half warp: whole ones in a dense matrix, and ragged rows with a stride."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K + pad), generator=g, device="cuda").to(torch.float32 if wide else torch.bfloat16)
    q = torch.full((M + 1, K), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M * -(-K // 128) + 1,), -1.0, device="cuda")
    V.vp_quant_fp8(x, V.VP_F32 if wide else V.VP_BF16, K + pad, M, K, q, s)
    torch.cuda.synchronize()
    assert (q[M] == 0x55).all() and s[-1] == -1.0
    assert_codes(q[:M].cpu().numpy(), f64(s[:-1]).reshape(M, -1), f64(x[:, :K]), 0.0, "many groups")


@pytest.mark.parametrize("M", [3, 400])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_add_rmsnorm_small_rows_with_zero_and_tiny_groups(V, M, weight, wide):
    """The row's factor is large; a group is zero, or its scale is at the floor."""
    rng = np.random.default_rng(M)
    K = 1280
    x = rng.standard_normal((M, K)) * np.array([1e-3, 1e-9, 1e-13])[np.arange(M) % 3][:, None]
    x[:, 256:384] = 0.0
    x[:, 640:768] = rng.standard_normal((M, 128)) * 1e-39
    x[:, 1024:1152] = rng.standard_normal((M, 128)) * 1e-38
    x[:, 1152:] = rng.standard_normal((M, 128)) * 1e-20
    x = f32(x) if wide else f32(x).to(torch.bfloat16)
    w = rng.uniform(0.5, 2, K)
    w[1152:] *= 1e-30  # products that fp32 loses before the row's factor
    w = f32(w) if weight else None
    _, q, s = run_norm(V, x, None, w, 1e-30, K)
    _, y = ref.add_rmsnorm(f64(x), None, f64(w) if weight else None, 1e-30)
    assert (s[:, 2] == 2.0 ** -126).all() and not (q[:, 256:384] & 127).any()
    if not weight:  # 5 * 1e-39 * 1e3 / 448 < 2^-126; a weight of 2 may exceed it
        assert (s[0::3, 5] == 2.0 ** -126).all()
    assert_codes(q, s, y, 40 * U, "small rows")


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("size", [1.0, 1e-22])
def test_add_rmsnorm_same_bits_with_and_without_h(V, wide, size):
    """Rare groups (ties under equal weights) and rows (squares outside fp32) are formed again from h or from the inputs."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((330, 1040)) * size
    x[:, ::7] = -0.0
    x = f32(x) if wide else f32(x).to(torch.bfloat16)
    w = torch.ones(1040, device="cuda")
    h, q, s = run_norm(V, x, None, w, 1e-30, 1040)
    _, q2, s2 = run_norm(V, x, None, w, 1e-30, 1040, h=None)
    assert np.array_equal(q, q2) and np.array_equal(s, s2)
    if not wide:
        x2 = x.clone()
        _, q3, s3 = run_norm(V, x2, None, w, 1e-30, 1040, h=x2)
        assert torch.equal(x2, h) and np.array_equal(q, q3) and np.array_equal(s, s3)


@pytest.mark.parametrize("M", [3, 400])
def test_add_rmsnorm_weights_without_a_value(V, M):
    """A NaN or an infinity among the weights reaches its group's scale in every row, and no other group."""
    rng = np.random.default_rng(M)
    K = 1280
    x, w = bf16(rng, (M, K)), rng.uniform(0.5, 2, K)
    x[1, 128 * 4 + 3] = 0.0
    w[128 * 4 + 3], w[128 * 9 + 5] = np.inf, np.nan
    _, q, s = run_norm(V, x, None, f32(w), 1e-6, K)
    with np.errstate(invalid="ignore"):
        _, y = ref.add_rmsnorm(f64(x), None, f64(f32(w)), 1e-6)
    ok = [b for b in range(10) if b not in (4, 9)]
    cols = np.concatenate([np.arange(b * 128, b * 128 + 128) for b in ok])
    assert_codes(q[:, cols], s[:, ok], y[:, cols], 40 * U, "weights without a value")
    v = ref.e4m3_value(q)
    assert np.isnan(s[:, 9]).all() and np.isnan(v[:, 128 * 9:]).all()
    inf = np.isinf(s[:, 4])
    assert inf.sum() == M - 1 and np.isnan(s[1, 4])  # 0 * inf
    assert np.isnan(v[inf, 128 * 4 + 3]).all() and not v[inf, 128 * 4 + 4:128 * 5].any()


@pytest.mark.parametrize("M", [5, 400])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_add_rmsnorm_weights_of_every_size(V, M, wide, in_place):
    """Groups whose products, or whose scales, leave the range that fp32 keeps exactly; a group of zero weights."""
    rng = np.random.default_rng(M + wide)
    K = 128 * 40
    x = f32(rng.standard_normal((M, K))) if wide else bf16(rng, (M, K))
    r = bf16(rng, (M, K))
    w = rng.uniform(0.5, 2, K).reshape(40, 128) * 10.0 ** np.linspace(-37, 37, 40)[:, None]
    w[7] = 0.0
    w = f32(w.reshape(-1))
    want_h, y = ref.add_rmsnorm(f64(x), bits16(r), f64(w), 1e-6)
    h, q, s = run_norm(V, x, r, w, 1e-6, K, h=r if in_place else None)
    if in_place:
        assert np.array_equal(bits16(h), want_h)
    assert_codes(q, s, y, 40 * U, "weights of every size")
    assert not (q[:, 7 * 128:8 * 128] & 127).any()


@pytest.mark.parametrize("M,K", [(4, 16384), (9, 2064), (700, 2064)])
@pytest.mark.parametrize("weight", ["random", "ones", "tenths"])
def test_add_rmsnorm_codes_round_once(V, M, K, weight):
    """The codes are those of the fp64 quotient but for ties (within 2^-36 of a border, which a weight of 24 bits
    times a value of 8 over another such product only meets by being one)."""
    rng = np.random.default_rng(M + K)
    x, r = bf16(rng, (M, K)), bf16(rng, (M, K))
    w = f32({"random": rng.uniform(-2, 2, K), "ones": np.ones(K), "tenths": np.full(K, 0.1)}[weight])
    _, q, _ = run_norm(V, x, r, w, 1e-6, K)
    _, y = ref.add_rmsnorm(f64(x), bits16(r), f64(w), 1e-6)
    want, off, border = nearest_codes(y, K)
    sure = (off > 2.0 ** -36) & (border > 2.0 ** -6)
    assert np.array_equal((q & 127)[sure], want[sure])
    assert np.abs((q & 127).astype(int) - want).max() <= 1


# ------------------------------------------------------------------ block-scaled linear
def codes(rng, shape):
    """Random finite e4m3 bytes, small magnitudes as likely as large ones."""
    c = rng.integers(0, 256, shape).astype(np.uint8)
    return np.where((c & 127) == 127, np.uint8(0x30), c)


def linear(V, xq, xs, wq, ws, y32, wsp=None, stream=None):
    M, K = xq.shape
    N = wq.shape[0]
    packed = torch.empty(V.vp_packed_bytes_fp8_block(N, K), dtype=torch.uint8, device="cuda")
    V.vp_pack_fp8_block(wq, N, K, packed, stream)
    y = torch.full((M + 1, N), 12345.0, dtype=torch.float32 if y32 else torch.bfloat16, device="cuda")
    if wsp is None:
        wsp = workspace(V.vp_linear_fp8_block_workspace_bytes(M, N, K))
    V.vp_linear_fp8_block(packed, ws, xq, xs, y, V.VP_F32 if y32 else V.VP_BF16, M, N, K, wsp, stream)
    torch.cuda.synchronize()
    assert V.vp_read_status(wsp) == V.VP_OK
    assert float(y[M].float().min()) == float(y[M].float().max())  # nothing behind the last row
    return y[:M]


def linear_case(seed, M, N, K):
    rng = np.random.default_rng(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    return (codes(rng, (M, K)), rng.uniform(0.5, 2, (M, kb)).astype(np.float32) * 1e-2, codes(rng, (N, K)),
            rng.uniform(0.5, 2, (nb, kb)).astype(np.float32) * 1e-3)


def dev_case(c):
    return torch.from_numpy(c[0]).cuda(), f32(c[1]), torch.from_numpy(c[2]).cuda(), f32(c[3])


SHAPES = [(1, 16, 16), (1, 16, 128), (3, 144, 144), (8, 5120, 1040), (8, 16, 17408), (15, 272, 256), (16, 256, 2560),
          (17, 640, 640), (32, 1040, 5120), (33, 2064, 384), (64, 128, 4096), (65, 144, 1152), (100, 1296, 528),
          (128, 256, 256), (129, 400, 272), (200, 5136, 640), (256, 256, 128), (257, 528, 2064), (500, 2560, 1296),
          (1025, 1040, 400), (2051, 4112, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_block(V, M, N, K):
    c = linear_case(M + N + K, M, N, K)
    y_ref, a_ref = ref.linear_block(*c)
    bound = 2 * (130 + -(-K // 128)) * U * a_ref + 1e-30
    y32 = f64(linear(V, *dev_case(c), True))
    assert_within(y32, y_ref, bound, f"linear fp32 {M}x{N}x{K}")
    y16 = linear(V, *dev_case(c), False)
    assert_within(f64(y16), y_ref, bound + 2.0 ** -8 * np.abs(y_ref), f"linear bf16 {M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 144, 272), (24, 528, 2064), (70, 400, 4112), (300, 1040, 1296)])
def test_linear_block_exact_on_dyadic_values(V, M, N, K):
    """Codes of small integers and power-of-two scales: every sum is an fp32 value, so bits agree."""
    rng = np.random.default_rng(K)
    ints = np.array([0, 0x38, 0x40, 0x44, 0xB8, 0xC0, 0xC4], np.uint8)  # 0, 1, 2, 3, -1, -2, -3
    xq, wq = ints[rng.integers(0, 7, (M, K))], ints[rng.integers(0, 7, (N, K))]
    kb, nb = -(-K // 128), -(-N // 128)
    xs = (2.0 ** rng.integers(-3, 2, (M, kb))).astype(np.float32)
    ws = (2.0 ** rng.integers(-3, 2, (nb, kb))).astype(np.float32)
    y = f64(linear(V, torch.from_numpy(xq).cuda(), f32(xs), torch.from_numpy(wq).cuda(), f32(ws), True))
    assert np.array_equal(y, ref.linear_block(xq, xs, wq, ws)[0])


def test_linear_block_repeats_and_shared_workspace(V):
    """One workspace of the largest call serves every shape in turn, without a reset, and a call gives the
    same bits alone, after others, and on another stream."""
    shapes = [(8, 5120, 1040), (200, 640, 2064), (3, 144, 144), (257, 528, 2064), (8, 16, 17408)]
    wsp = workspace(max(V.vp_linear_fp8_block_workspace_bytes(*s) for s in shapes))
    cases = [dev_case(linear_case(7, *s)) for s in shapes]
    alone = [linear(V, *c, True) for c in cases]
    for _ in range(2):
        for c, y in zip(cases, alone):
            assert torch.equal(linear(V, *c, True, wsp=wsp), y)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, y in zip(cases, alone):
        assert torch.equal(linear(V, *c, True, wsp=wsp, stream=st), y)


def test_linear_block_nan_stays_in_its_row_and_column(V):
    M, N, K = 40, 272, 400
    c = dev_case(linear_case(1, M, N, K))
    good = linear(V, *c, True)
    c[0][7, 300], c[2][260, 3] = 0x7F, 0xFF
    c[1][9, 0] = float("inf")
    y = linear(V, *c, True)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[7], bad[:, 260] = True, True
    assert bool(torch.isnan(y[7]).all()) and bool(torch.isnan(y[:, 260]).all())
    assert not bool(torch.isfinite(y[9]).any())
    bad[9] = True
    assert torch.equal(y[~bad], good[~bad])


def test_linear_block_graph_replays_with_new_inputs(V):
    M, N, K = 20, 400, 1296
    a, b = dev_case(linear_case(1, M, N, K)), dev_case(linear_case(2, M, N, K))
    want = linear(V, *b[:2], *a[2:], True)
    packed = torch.empty(V.vp_packed_bytes_fp8_block(N, K), dtype=torch.uint8, device="cuda")
    V.vp_pack_fp8_block(a[2], N, K, packed)
    xq, xs = a[0].clone(), a[1].clone()
    y = torch.empty((M, N), device="cuda")
    wsp = workspace(V.vp_linear_fp8_block_workspace_bytes(M, N, K))
    call = lambda: V.vp_linear_fp8_block(packed, a[3], xq, xs, y, V.VP_F32, M, N, K, wsp)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    xq.copy_(b[0])
    xs.copy_(b[1])
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


# ------------------------------------------------------------------ paged append
class Paged:
    """Random caches and a page table in which every (sequence, page) has a page of its own."""

    def __init__(self, V, seed, S, max_pages, P, Hkv, D, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.S, self.P, self.Hkv, self.D, self.max_pages = S, P, Hkv, D, max_pages
        self.n = S * max_pages + spare
        self.k = torch.randn((self.n, Hkv, P, D), generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((self.n, Hkv, P, D), generator=g, device="cuda").to(torch.bfloat16)
        self.table = np.random.default_rng(seed).permutation(self.n)[:S * max_pages].reshape(S, max_pages).astype(np.int32)
        self.pages = i32(self.table)
        self.V = V

    def desc(self):
        return self.V.vp_paged_cache(self.k, self.v, self.pages, self.n, self.P, self.max_pages, self.Hkv, self.D)


def freqs(rot, base=10000.0):
    return [base ** (-2.0 * j / rot) for j in range(rot // 2)]


@pytest.mark.parametrize("D,Hq,Hkv,P,rot,inter,norm", [
    (256, 24, 4, 64, 256, True, True),    # this model family's attention
    (256, 6, 1, 16, 64, False, True),     # a quarter of the head rotates
    (128, 32, 8, 16, 128, False, False),
    (128, 5, 5, 32, 96, False, True),     # pairs that do not fill the lanes evenly
    (64, 8, 2, 128, 64, True, False),
    (64, 3, 1, 64, 16, False, True),
    (128, 4, 2, 64, 0, True, False),      # no rotation: a copy
])
def test_append(V, D, Hq, Hkv, P, rot, inter, norm):
    rng = np.random.default_rng(D + rot)
    rows, ctx = [1, 0, P + 3, 2, 1], [0, 5, P - 2, 3 * P - 1, 2 * P]  # rows of none, over page ends
    S, T, pad = len(rows), sum(rows), 2
    start = np.cumsum([1] + rows)  # row 0 is padding, and so is the last
    M = T + pad
    p = Paged(V, D + P, S, 5, P, Hkv, D)
    ld = (Hq + 2 * Hkv) * D + 24
    x = bf16(rng, (M, ld))
    q, k, v = x[:, :Hq * D], x[:, Hq * D:(Hq + Hkv) * D], x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D]
    v[3, 5] = float("nan")
    qn = f32(rng.uniform(0.5, 1.5, D)) if norm else None
    kn = f32(rng.uniform(0.5, 1.5, D)) if norm else None
    rope = V.vp_rope(freqs(rot), inter) if rot else None
    k0, v0 = p.k.clone(), p.v.clone()
    q_out = torch.full((M, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kv_len, status = i32([-9] * S), i32([0])
    V.vp_paged_append(p.desc(), q, ld, k, ld, v, ld, qn, kn, 1e-6, rope, i32(start), i32(ctx), S, M, Hq, q_out, kv_len,
                      status)
    torch.cuda.synchronize()
    assert int(status) == 0 and kv_len.tolist() == [a + b for a, b in zip(ctx, rows)]
    assert bool((q_out[0] == 7.0).all()) and bool((q_out[-1] == 7.0).all())  # padding rows
    seq = np.repeat(np.arange(S), rows)
    pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, rows)])
    fr = freqs(rot) if rot else []
    for name, src, w, H in (("q", q, qn, Hq), ("k", k, kn, Hkv)):
        xin = f64(src[1:1 + T]).reshape(T, H, D)
        want, mag = ref.norm_rope(xin, f64(w) if norm else None, 1e-6, pos, fr, inter)
        if name == "q":
            got = f64(q_out[1:1 + T])
        else:
            got = f64(p.k[p.table[seq, pos // P], :, pos % P])
        assert_within(got, want, 2.0 ** -8 * np.abs(want) + (32 * U * mag if (norm or rot) else 0), f"append {name}")
        if not norm and rot < D:
            assert np.array_equal(got[..., rot:], xin[..., rot:])
    at = torch.from_numpy(p.table[seq, pos // P]).cuda().long(), torch.from_numpy(pos % P).cuda()
    assert torch.equal(p.v[at[0], :, at[1]].view(torch.int16), v[1:1 + T].reshape(T, Hkv, D).view(torch.int16))
    # nothing else in the caches changed
    p.k[at[0], :, at[1]], p.v[at[0], :, at[1]] = k0[at[0], :, at[1]], v0[at[0], :, at[1]]
    assert torch.equal(p.k.view(torch.int16), k0.view(torch.int16)) and torch.equal(p.v.view(torch.int16), v0.view(torch.int16))


def test_append_one_row_per_sequence_equals_ragged_and_in_place(V):
    rng = np.random.default_rng(0)
    S, Hq, Hkv, D, P = 70, 6, 2, 128, 32
    ctx = rng.integers(0, 4 * P, S)
    q, k, v = bf16(rng, (S, Hq, D)), bf16(rng, (S, Hkv, D)), bf16(rng, (S, Hkv, D))
    rope, w = V.vp_rope(freqs(128), False), f32(rng.uniform(0.5, 1.5, D))
    res = []
    for start in (None, i32(np.arange(S + 1))):
        p = Paged(V, 1, S, 4, P, Hkv, D)
        out = torch.empty_like(q)
        V.vp_paged_append(p.desc(), q, Hq * D, k, Hkv * D, v, Hkv * D, w, w, 1e-6, rope, start, i32(ctx), S, S, Hq, out)
        res.append((out, p.k, p.v))
    assert all(torch.equal(a, b) for a, b in zip(*res))
    p = Paged(V, 1, S, 4, P, Hkv, D)
    mine = q.clone()
    V.vp_paged_append(p.desc(), mine, Hq * D, k, Hkv * D, v, Hkv * D, w, w, 1e-6, rope, None, i32(ctx), S, S, Hq, mine)
    assert torch.equal(mine, res[0][0])
    p = Paged(V, 1, S, 4, P, Hkv, D)  # keys and values alone
    V.vp_paged_append(p.desc(), None, 0, k, Hkv * D, v, Hkv * D, w, w, 1e-6, rope, None, i32(ctx), S, S, 0, None)
    assert torch.equal(p.k, res[0][1]) and torch.equal(p.v, res[0][2])


def test_append_far_positions(V):
    """Positions near 2^27 in a table of shared pages: the angle keeps its digits."""
    rng = np.random.default_rng(5)
    S, Hq, Hkv, D, P = 4, 2, 1, 64, 128
    max_pages = 1 << 20
    p = Paged(V, 2, S, 1, P, Hkv, D)
    table = torch.full((S, max_pages), 0, dtype=torch.int32, device="cuda")
    ctx = np.array([(1 << 27) - 1, 100_000_007, 1_000_003, 131_071])
    for s in range(S):
        table[s, ctx[s] // P] = s + 1
    p.pages, p.max_pages = table, max_pages
    q, k, v = bf16(rng, (S, Hq, D)), bf16(rng, (S, Hkv, D)), bf16(rng, (S, Hkv, D))
    out = torch.empty_like(q)
    fr = freqs(64, 1e6)
    V.vp_paged_append(p.desc(), q, Hq * D, k, D, v, D, None, None, 0.0, V.vp_rope(fr, True), None, i32(ctx), S, S, Hq, out)
    for got, src, H in ((f64(out), q, Hq), (f64(p.k[torch.arange(S) + 1, :, torch.from_numpy(ctx % P)]), k, Hkv)):
        want, mag = ref.norm_rope(f64(src), None, 0, ctx, fr, True)
        # the oracle's own angle, position * frequency in fp64, is off by up to 2^27 2^-53 more
        assert_within(got, want, 2.0 ** -8 * np.abs(want) + (32 * U + 2.0 ** -26) * mag, "far positions")


def test_append_reports_bad_rows_and_skips_them(V):
    rng = np.random.default_rng(6)
    S, Hq, Hkv, D, P = 6, 2, 1, 64, 16
    ctx = [3, -1, 32, 5, 5, 2147483647]  # good, negative, beyond the table, bad page, page too high, largest
    p = Paged(V, 3, S, 2, P, Hkv, D)
    p.pages[3, 0], p.pages[4, 0] = -1, p.n
    k0, v0 = p.k.clone(), p.v.clone()
    q, k, v = bf16(rng, (S, Hq, D)), bf16(rng, (S, Hkv, D)), bf16(rng, (S, Hkv, D))
    out, status, kv_len = torch.full_like(q, 5.0), i32([0]), i32([0] * S)
    V.vp_paged_append(p.desc(), q, Hq * D, k, D, v, D, None, None, 0.0, None, None, i32(ctx), S, S, Hq, out, kv_len, status)
    assert int(status) == V.VP_ERR_SHAPE
    assert kv_len.tolist() == [4, 0, 33, 6, 6, 2147483647]
    assert torch.equal(out[0], q[0]) and not bool(out[1:].any())
    pg = int(p.table[0, 0])
    assert torch.equal(p.k[pg, :, 3], k[0]) and torch.equal(p.v[pg, :, 3], v[0])
    p.k[pg, :, 3], p.v[pg, :, 3] = k0[pg, :, 3], v0[pg, :, 3]
    assert torch.equal(p.k, k0) and torch.equal(p.v, v0)
    status.zero_()  # rows that the call does not have
    V.vp_paged_append(p.desc(), q, Hq * D, k, D, v, D, None, None, 0.0, None, i32([0, 1, 1, 1, 1, 1, 9]), i32([0] * S), S, S,
                      Hq, out, None, status)
    assert int(status) == V.VP_ERR_SHAPE


# ------------------------------------------------------------------ paged attention
def attend(V, p, q, kv_len, scale, gate=None, want_lse=True, ws=None, expect=0, stream=None):
    S, Hq, D = q.shape
    out = torch.full((S + 1, Hq, D), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((S + 1, Hq), 9.0, device="cuda") if want_lse else None
    ws = workspace(V.vp_paged_attention_workspace_bytes(S, Hq, p.Hkv, D)) if ws is None else ws
    V.vp_paged_attention(p.desc(), q, i32(kv_len), S, Hq, scale, gate, out, lse, ws, stream)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == expect
    assert bool((out[S] == 9.0).all()) and (lse is None or bool((lse[S] == 9.0).all()))
    return out[:S], lse[:S] if want_lse else None


def check_attend(V, p, q, kv_len, scale, gate=None, k=None, v=None, expect=0, what=""):
    out, lse = attend(V, p, q, kv_len, scale, gate, expect=expect)
    S, Hq, D = q.shape
    table = p.pages.cpu().numpy()
    want, mag, want_lse, dot = ref.paged_attention(f64(q), f64(p.k if k is None else k), f64(p.v if v is None else v), table,
                                                   kv_len, scale, f64(gate) if gate is not None else None)
    e = (2 * D + 4) * U * dot
    n = np.maximum(np.asarray(kv_len, np.float64), 1)[:, None]
    bound = (np.expm1(2 * e) + 2.0 ** -16 + n * U)[..., None] * mag + 2.0 ** -8 * np.abs(want) + 1e-37
    assert_within(f64(out), want, bound, "attention " + what)
    fin = np.isfinite(want_lse)
    got = f64(lse)
    assert np.array_equal(np.isneginf(got), ~fin)
    assert_within(got[fin], want_lse[fin], (e + 2.0 ** -16 + n * U + 4 * U * np.abs(np.where(fin, want_lse, 0)))[fin], "lse " + what)
    return out, lse


@pytest.mark.parametrize("D,Hq,Hkv,P,lens", [
    (256, 24, 4, 64, [1]),
    (256, 24, 4, 64, [0, 1, 15, 16, 17, 63, 64, 65, 700]),
    (256, 6, 1, 16, [2500]),               # one sequence and head over every CTA
    (256, 16, 1, 32, [333, 31]),           # a group of 16
    (256, 9, 1, 128, [257, 128]),          # a group of 9
    (128, 32, 8, 16, [100, 0, 1, 999, 16, 48]),
    (128, 5, 5, 32, [33, 64, 1]),          # groups of one
    (128, 48, 4, 128, [1000, 129]),
    (64, 8, 2, 128, [128, 1, 385, 0, 64]),
    (64, 14, 1, 16, [555, 17]),
    (64, 11, 11, 64, [70, 200]),
])
def test_attention(V, D, Hq, Hkv, P, lens):
    rng = np.random.default_rng(D + Hq)
    S = len(lens)
    p = Paged(V, Hq + P, S, max(1, -(-max(lens) // P)) + 1, P, Hkv, D)
    q, gate = bf16(rng, (S, Hq, D), 1.5), bf16(rng, (S, Hq, D), 2.0)
    a, lse_a = check_attend(V, p, q, lens, D ** -0.5, gate, what=f"{D} {Hq}/{Hkv} {P}")
    b, _ = check_attend(V, p, q, lens, -0.3 * D ** -0.5, None, what="no gate, negative scale")
    again, lse_b = attend(V, p, q, lens, D ** -0.5, gate)
    assert torch.equal(a, again) and torch.equal(lse_a, lse_b)
    without, _ = attend(V, p, q, lens, D ** -0.5, gate, want_lse=False)
    assert torch.equal(a, without)


@pytest.mark.parametrize("S,Hq,Hkv,D,P,top", [(70, 8, 2, 128, 16, 600), (300, 6, 3, 64, 32, 90), (1000, 1, 1, 64, 16, 40),
                                              (33, 24, 4, 256, 64, 400)])
def test_attention_many_ragged_sequences(V, S, Hq, Hkv, D, P, top):
    rng = np.random.default_rng(S)
    lens = rng.integers(0, top + 1, S)
    lens[0], lens[-1] = top, 0
    p = Paged(V, S, S, -(-top // P), P, Hkv, D)
    check_attend(V, p, bf16(rng, (S, Hq, D), 1.5), lens, D ** -0.5, what=f"{S} sequences")


def test_attention_what_lies_behind_the_end_has_no_effect(V):
    """Infinities and NaN in the slots behind kv_len, in the pages behind the last one, and in page ids
    there; a page shared by two sequences."""
    rng = np.random.default_rng(8)
    for D, P in ((256, 64), (128, 16), (64, 128)):
        lens = [P + 5, 1, 2 * P]
        p = Paged(V, 9, 3, 4, P, 2, D)
        p.pages[1, 0] = p.pages[0, 0]
        k, v = p.k.clone(), p.v.clone()
        for s, n in ((0, P + 5), (2, 2 * P)):
            for j in range(4):
                lo = min(max(n - j * P, 0), P)
                pg = int(p.table[s, j])
                p.k[pg, :, lo:], p.v[pg, :, lo:] = float("nan"), float("inf")
        p.pages[0, 3], p.pages[1, 1], p.pages[2, 2] = -5, 1 << 30, -1
        q = bf16(rng, (3, 6, D), 1.5)
        check_attend(V, p, q, lens, D ** -0.5, k=k, v=v, what=f"behind the end, D={D}")


def test_attention_reports_bad_lengths_and_pages(V):
    rng = np.random.default_rng(10)
    P, D = 32, 128
    p = Paged(V, 11, 5, 4, P, 2, D)
    p.pages[3, 1], p.pages[4, 0] = p.n, -1
    q = bf16(rng, (5, 4, D), 1.5)
    lens = [100, -1, 4 * P + 1, 100, 20]  # good, negative, beyond the table, a bad page inside, only a bad page
    out, lse = check_attend(V, p, q, lens, D ** -0.5, expect=V.VP_ERR_SHAPE, what="bad pages")
    assert not bool(out[1].any()) and not bool(out[2].any()) and not bool(out[4].any())
    assert bool(torch.isneginf(lse[[1, 2, 4]]).all())


def test_attention_extreme_values(V):
    """Values over bf16's range per head, scores far apart (one key takes all the weight), equal scores, and
    a key of infinities (its NaN or infinite score reaches its own sequence only)."""
    rng = np.random.default_rng(12)
    P, D = 64, 256
    p = Paged(V, 13, 2, 6, P, 4, D)
    p.v *= torch.tensor([1e30, 1e6, 1e-30, 3.0], device="cuda")[None, :, None, None].to(torch.bfloat16)
    q = bf16(rng, (2, 24, D), 1.5)
    q[:, 12:] *= 40.0
    q[1, :6] = 0.0
    check_attend(V, p, q, [300, 200], D ** -0.5, what="extreme values")
    good, _ = attend(V, p, q, [300, 200], D ** -0.5)
    p.k[int(p.table[0, 2]), 0, 7, 3] = float("inf")
    out, _ = attend(V, p, q, [300, 200], D ** -0.5)
    assert torch.equal(out[1], good[1]) and torch.equal(out[0, 6:], good[0, 6:])
    # a head whose q element there is positive has an infinite score: its softmax has no value
    pos = q[0, :6, 3] > 0
    assert bool(torch.isnan(out[0, :6][pos]).all())
    assert bool(torch.isfinite(out[0, :6][q[0, :6, 3] < 0]).all())


def test_attention_offsets_beyond_32_bits(V):
    """Pages behind 2^32 elements of the cache (append and attention), 8.6 GB each for keys and values."""
    Hkv, P, D = 4, 64, 256
    n = (1 << 32) // (Hkv * P * D) + 8
    k, v = (torch.empty((n, Hkv, P, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rng = np.random.default_rng(14)
    p = Paged(V, 15, 1, 2, P, Hkv, D)
    small_k, small_v, small_pages = p.k, p.v, p.table.copy()
    high = [n - 1, n - 4]
    for j in range(2):
        k[high[j]], v[high[j]] = small_k[int(small_pages[0, j])], small_v[int(small_pages[0, j])]
    q = bf16(rng, (1, 24, D), 1.5)
    nk, nv = bf16(rng, (1, Hkv, D)), bf16(rng, (1, Hkv, D))
    res = []
    for kk, vv, tab, np_ in ((small_k, small_v, small_pages, p.n), (k, v, np.array([high], np.int32), n)):
        p.k, p.v, p.pages, p.n = kk, vv, i32(tab), np_
        q_out = torch.empty_like(q)
        kv_len = i32([0])
        V.vp_paged_append(p.desc(), q, 24 * D, nk, Hkv * D, nv, Hkv * D, None, None, 0.0, V.vp_rope(freqs(256), True), None,
                          i32([100]), 1, 1, 24, q_out, kv_len)
        res.append(attend(V, p, q_out, [101], 0.0625))
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


def test_attention_shared_workspace_streams_and_graph(V):
    """One workspace, calls of other sizes before, a side stream, and a captured decode step (append, then
    attention with the lengths that the append wrote) replayed as the sequences grow."""
    rng = np.random.default_rng(16)
    S, Hq, Hkv, D, P = 3, 8, 2, 128, 16
    p = Paged(V, 17, S, 40, P, Hkv, D)
    big = Paged(V, 18, 9, 20, 32, 4, 256)
    ws = workspace(max(V.vp_paged_attention_workspace_bytes(9, 24, 4, 256), V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D)))
    qb, q = bf16(rng, (9, 24, 256)), bf16(rng, (S, Hq, D), 1.5)
    lens = [600, 5, 333]
    alone, _ = attend(V, p, q, lens, D ** -0.5)
    for _ in range(2):
        attend(V, big, qb, [640] * 9, 0.0625, ws=ws)
        assert torch.equal(attend(V, p, q, lens, D ** -0.5, ws=ws)[0], alone)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.equal(attend(V, p, q, lens, D ** -0.5, ws=ws, stream=st)[0], alone)
    # the captured step: two appends and attentions, the lengths passed from one to the next on the device
    k, v = bf16(rng, (S, Hkv, D)), bf16(rng, (S, Hkv, D))
    len_a, len_b = i32([600, 5, 333]), i32([0] * S)
    out, q_rot = torch.empty_like(q), torch.empty_like(q)
    rope = V.vp_rope(freqs(D), False)
    desc = p.desc()

    def half(src, dst):
        V.vp_paged_append(desc, q, Hq * D, k, Hkv * D, v, Hkv * D, None, None, 0.0, rope, None, src, S, S, Hq, q_rot, dst)
        V.vp_paged_attention(desc, q_rot, dst, S, Hq, D ** -0.5, None, out, None, ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        half(len_a, len_b)
        half(len_b, len_a)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert len_a.tolist() == [606, 11, 339]
    assert V.vp_read_status(ws) == V.VP_OK
    check = attend(V, p, q_rot, [606, 11, 339], D ** -0.5)[0]
    assert torch.equal(check, out)
    check_attend(V, p, q_rot, [606, 11, 339], D ** -0.5, what="after replays")


@pytest.mark.parametrize("D,Hq,Hkv,P,lens", [
    (256, 8, 1, 128, [40000]),             # one head over every CTA: its parts come in several rounds
    (64, 16, 1, 16, [70001]),              # the same above 8 heads
    (128, 16, 2, 32, [9000, 3, 0, 5000]),  # long and short ones together
    (128, 64, 8, 16, [1500] * 12),         # more (sequence, head)s than half the CTAs: runs over their borders
    (64, 24, 24, 64, [900, 1, 64, 333, 2000, 0, 77]),
])
def test_attention_every_way_of_cutting(V, D, Hq, Hkv, P, lens):
    rng = np.random.default_rng(len(lens) + D)
    S = len(lens)
    p = Paged(V, 31, S, -(-max(lens) // P), P, Hkv, D)
    q, gate = bf16(rng, (S, Hq, D), 1.5), bf16(rng, (S, Hq, D), 2.0)
    a, lse = check_attend(V, p, q, lens, D ** -0.5, gate, what=f"{S} x {max(lens)}")
    b, lse_b = attend(V, p, q, lens, D ** -0.5, gate)
    assert torch.equal(a, b) and torch.equal(lse, lse_b)


def test_one_workspace_for_calls_of_every_shape(V):
    """A workspace of the largest size serves attention and linear calls of any shapes in turn, without a
    reset: the counters of one call are never another one's data."""
    rng = np.random.default_rng(33)
    calls = []
    for S, Hq, Hkv, D, P, top in ((1000, 4, 2, 64, 16, 70), (1, 8, 1, 256, 64, 9000), (300, 12, 4, 128, 32, 500),
                                  (4, 24, 4, 256, 64, 700)):
        p = Paged(V, S, S, -(-top // P), P, Hkv, D)
        lens = rng.integers(0, top + 1, S)
        lens[0] = top
        q = bf16(rng, (S, Hq, D), 1.5)
        calls.append((V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D),
                      lambda ws, p=p, q=q, lens=lens, D=D: attend(V, p, q, lens, D ** -0.5, ws=ws)[0]))
    for M, N, K in ((8, 2560, 4096), (300, 1040, 2064), (100, 640, 640)):
        c = dev_case(linear_case(M, M, N, K))
        calls.append((V.vp_linear_fp8_block_workspace_bytes(M, N, K), lambda ws, c=c: linear(V, *c, True, wsp=ws)))
    alone = [f(workspace(n)) for n, f in calls]
    ws = workspace(max(n for n, _ in calls))
    for _ in range(2):
        for (_, f), want in zip(calls, alone):
            assert torch.equal(f(ws), want)
    for i in (6, 2, 5, 0, 4, 3, 1):
        assert torch.equal(calls[i][1](ws), alone[i])


def test_calls_on_two_streams_at_once(V):
    """Independent calls overlap: a linear of each kind beside attention, each with its own workspace."""
    rng = np.random.default_rng(34)
    p = Paged(V, 35, 40, 16, 64, 4, 256)
    q, lens = bf16(rng, (40, 24, 256), 1.5), i32([1000] * 40)
    want_o, _ = attend(V, p, q, [1000] * 40, 0.0625)
    shapes = [(8, 5120, 4096), (100, 2560, 4096), (1500, 2560, 2048)]
    cases = [dev_case(linear_case(1, *s)) for s in shapes]
    want = [linear(V, *c, True) for c in cases]
    packs, ys, lws = [], [], []
    for c, (M, N, K) in zip(cases, shapes):
        packs.append(torch.empty(V.vp_packed_bytes_fp8_block(N, K), dtype=torch.uint8, device="cuda"))
        V.vp_pack_fp8_block(c[2], N, K, packs[-1])
        ys.append(torch.empty((M, N), device="cuda"))
        lws.append(workspace(V.vp_linear_fp8_block_workspace_bytes(M, N, K)))
    out = torch.empty_like(q)
    aws = workspace(V.vp_paged_attention_workspace_bytes(40, 24, 4, 256))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    desc = p.desc()
    for _ in range(10):
        V.vp_paged_attention(desc, q, lens, 40, 24, 0.0625, None, out, None, aws, stream=s1)
        for pk, c, y, w, (M, N, K) in zip(packs, cases, ys, lws, shapes):
            V.vp_linear_fp8_block(pk, c[3], c[0], c[1], y, V.VP_F32, M, N, K, w, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(out, want_o) and all(torch.equal(a, b) for a, b in zip(ys, want))
    assert V.vp_read_status(aws) == V.VP_OK and all(V.vp_read_status(w) == V.VP_OK for w in lws)


@pytest.mark.parametrize("S", [100, 128, 129, 256, 257, 700])
def test_append_finds_the_sequence_of_every_row(V, S):
    """Row offsets with empty sequences and padding at both ends, over each way of looking a row up."""
    rng = np.random.default_rng(S)
    rows = rng.integers(0, 4, S)
    ctx = rng.integers(0, 30, S)
    start = 3 + np.concatenate([[0], np.cumsum(rows)])
    T = int(rows.sum())
    M, Hkv, D, P = T + 8, 2, 64, 16
    p = Paged(V, S, S, 3, P, Hkv, D)
    k, v = bf16(rng, (M, Hkv, D)), bf16(rng, (M, Hkv, D))
    want_k, want_v = p.k.clone(), p.v.clone()
    seq = np.repeat(np.arange(S), rows)
    pos = np.repeat(ctx, rows) + np.concatenate([np.arange(n) for n in rows])
    pg, sl = torch.from_numpy(p.table[seq, pos // P]).cuda().long(), torch.from_numpy(pos % P).cuda()
    want_k[pg, :, sl], want_v[pg, :, sl] = k[3:3 + T], v[3:3 + T]
    kv_len, status = i32([0] * S), i32([0])
    V.vp_paged_append(p.desc(), None, 0, k, Hkv * D, v, Hkv * D, None, None, 0.0, None, i32(start), i32(ctx), S, M, 0, None,
                      kv_len, status)
    assert torch.equal(p.k, want_k) and torch.equal(p.v, want_v)
    assert kv_len.tolist() == (ctx + rows).tolist() and int(status) == 0


# ------------------------------------------------------------------ together
def test_layer_of_a_served_step(V):
    """One attention layer as it is used: a prompt of two sequences, then two single-token steps.  Every
    operator is checked against its definition from the device's own input to it."""
    rng = np.random.default_rng(20)
    H, Hq, Hkv, D, P, S = 640, 6, 2, 128, 16, 2
    N = (Hq + 2 * Hkv) * D
    p = Paged(V, 21, S, 6, P, Hkv, D)
    wqkv = linear_case(22, 1, N, H)[2:]
    wo = linear_case(23, 1, H, Hq * D)[2:]
    packs = []
    for w, _ in (wqkv, wo):
        packs.append(torch.empty(V.vp_packed_bytes_fp8_block(*w.shape), dtype=torch.uint8, device="cuda"))
        V.vp_pack_fp8_block(torch.from_numpy(w).cuda(), *w.shape, packs[-1])
    nw, qn = f32(rng.uniform(0.5, 1.5, H)), f32(rng.uniform(0.5, 1.5, D))
    rope, fr = V.vp_rope(freqs(D), False), freqs(D)
    ctx = np.zeros(S, np.int64)
    aws = workspace(V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D))
    for rows in ([37, 20], [1, 1], [1, 1]):
        M = sum(rows)
        resid, x = bf16(rng, (M, H)), f32(rng.standard_normal((M, H)))
        h, q8, s8 = run_norm(V, x, resid, nw, 1e-6, H)
        want_h, y = ref.add_rmsnorm(f64(x), bits16(resid), f64(nw), 1e-6)
        assert np.array_equal(bits16(h), want_h)
        assert_codes(q8, s8, y, 40 * U, "layer norm")
        lws = workspace(max(V.vp_linear_fp8_block_workspace_bytes(M, N, H), V.vp_linear_fp8_block_workspace_bytes(M, H, Hq * D)))
        qkv = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        V.vp_linear_fp8_block(packs[0], f32(wqkv[1]), torch.from_numpy(q8).cuda(), f32(s8), qkv, V.VP_BF16, M, N, H, lws)
        want, a = ref.linear_block(q8, s8, *wqkv)
        assert_within(f64(qkv), want, 2 * (130 + 5) * U * a + 2.0 ** -8 * np.abs(want), "layer qkv")
        q_out, kv_len, status = torch.empty((M, Hq, D), dtype=torch.bfloat16, device="cuda"), i32([0] * S), i32([0])
        V.vp_paged_append(p.desc(), qkv, N, qkv[:, Hq * D:], N, qkv[:, (Hq + Hkv) * D:], N, qn, qn, 1e-6, rope,
                          i32(np.cumsum([0] + rows)), i32(ctx), S, M, Hq, q_out, kv_len, status)
        pos = np.concatenate([c + np.arange(n) for c, n in zip(ctx, rows)])
        want, mag = ref.norm_rope(f64(qkv[:, :Hq * D]).reshape(M, Hq, D), f64(qn), 1e-6, pos, fr, False)
        assert_within(f64(q_out), want, 2.0 ** -8 * np.abs(want) + 32 * U * mag, "layer q")
        ctx = ctx + rows
        assert kv_len.tolist() == ctx.tolist() and int(status) == 0
        last = torch.from_numpy(np.cumsum(rows) - 1).cuda()  # the newest token of each sequence
        out, _ = check_attend(V, p, q_out[last].contiguous(), ctx, D ** -0.5, what="layer")
        o8 = torch.empty((S, Hq * D), dtype=torch.uint8, device="cuda")
        os_ = torch.empty((S, Hq), device="cuda")
        V.vp_quant_fp8(out, V.VP_BF16, Hq * D, S, Hq * D, o8, os_)
        assert_codes(o8.cpu().numpy(), f64(os_), f64(out).reshape(S, -1), 0.0, "layer o input")
        yo = torch.empty((S, H), device="cuda")
        V.vp_linear_fp8_block(packs[1], f32(wo[1]), o8, os_, yo, V.VP_F32, S, H, Hq * D, lws)
        want, a = ref.linear_block(o8.cpu().numpy(), f64(os_), *wo)
        assert_within(f64(yo), want, 2 * (130 + 6) * U * a, "layer o")
        assert V.vp_read_status(lws) == V.VP_OK and V.vp_read_status(aws) == V.VP_OK
