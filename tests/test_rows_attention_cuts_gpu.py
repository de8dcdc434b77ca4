"""Nothing is lost or counted twice where the work is cut: values that mark the position, in groups of 16 keys (the smallest page), so
that a group more or less changes four or more columns of a row by several times the tolerance
(test_rows_attention_cuts_cpu.py).  With random values a lost block of a long context hides behind the rounding of the weights."""
import numpy as np
import pytest
import torch

from helpers import workspace
from test_rows_attention_gpu import Cache, buffers, check, want_of
from test_served_layer_gpu import bf16, f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def V():
    from weight_streaming_gb300 import _lib
    return _lib


# positions in all, new rows
CASES = [(256, 6, 1, 1, [40000]), (128, 4, 1, 8, [30000]), (64, 2, 1, 300, [20000]), (256, 2, 1, 200, [9000]), (64, 1, 1, 1, [25000]),
         (128, 4, 2, 1, [9000, 17, 300, 12345, 64]), (256, 8, 2, 5, [7000, 5, 3001]), (128, 16, 1, 40, [6000, 2300]), (64, 64, 1, 2, [8000, 130]),
         (256, 6, 1, 90, [5000, 90, 1234])]


def marks(t, D):
    """The value of position t: its group's column."""
    return (t[:, None] // 16 % D == np.arange(D)).astype(np.float64)


def queries(seed, n, Hq, D):
    """Scores that spread by about 1/2: no position has much more weight than another."""
    return bf16(np.random.default_rng(seed), (n, Hq, D), 0.5)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hkv,n,lens", CASES)
def test_every_position_once(V, D, Hq, Hkv, n, lens, fp8):
    S, P = len(lens), 16
    c, M = Cache(V, 3, S, -(-max(lens) // P), P, Hkv, D, fp8), S * n
    for s in range(S):
        m = torch.from_numpy(marks(np.arange(c.max_pages * P), D)).cuda().view(c.max_pages, 1, P, D)
        pg = torch.from_numpy(c.table[s]).cuda().long()
        c.v[pg] = (m * 0x38).to(torch.uint8).expand(-1, Hkv, -1, -1) if fp8 else m.to(torch.bfloat16).expand(-1, Hkv, -1, -1)
    if fp8:
        c.vs.fill_(127)
    q = queries(n, M, Hq, D)
    out, lse, _ = buffers(M, Hq, D, False)
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    c.attend(q, i32(np.arange(S + 1) * n), i32(lens), M, Hq, D ** -0.5, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    kv = [c.values(s, lens[s]) for s in range(S)]
    want, m = want_of(q, np.arange(S + 1) * n, [x[0] for x in kv], [x[1] for x in kv], [x - n for x in lens], None, D ** -0.5, None)
    check(out, lse, want, m, D, f"cuts {D} {fp8}")


@pytest.mark.parametrize("D,Hq,Hkv,rows", [(64, 2, 1, [4000]), (128, 4, 2, [2100, 1, 300]), (256, 4, 2, [1500, 700]), (256, 1, 1, [3500]),
                                           (128, 1, 1, [100] * 9), (64, 1, 1, [120, 128] * 4), (256, 1, 1, [128] * 7)])
def test_every_position_of_a_prompt_once(V, D, Hq, Hkv, rows):
    M, S, start = sum(rows), len(rows), np.cumsum([0] + rows)
    q, k = queries(1, M, Hq, D), bf16(np.random.default_rng(2), (M, Hkv, D))
    v = torch.from_numpy(np.concatenate([marks(np.arange(n), D) for n in rows])).cuda().to(torch.bfloat16)
    v = v[:, None].expand(M, Hkv, D).contiguous()
    out, lse, _ = buffers(M, Hq, D, False)
    ws = workspace(V.vp_prompt_attention_workspace_bytes(S, M, Hq, Hkv, D))
    V.vp_prompt_attention(q, Hq * D, k, Hkv * D, v, Hkv * D, i32(start), S, M, Hq, Hkv, D, D ** -0.5, None, out, lse, ws)
    torch.cuda.synchronize()
    assert V.vp_read_status(ws) == V.VP_OK
    part = [slice(a, b) for a, b in zip(start, start[1:])]
    want, m = want_of(q, start, [f64(k[p]) for p in part], [f64(v[p]) for p in part], [0] * S, None, D ** -0.5, None)
    check(out, lse, want, m, D, f"prompt cuts {D}")
