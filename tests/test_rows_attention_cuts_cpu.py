"""The bound of test_rows_attention_cuts_gpu.py rejects outputs that lack a group of 16 keys or count one twice, wherever it lies, and
takes the definition's own."""
import numpy as np
import pytest
import torch

from oracle import served_layer as ref
from test_rows_attention_cuts_gpu import CASES, marks
from test_rows_attention_gpu import check, want_of


def result(q, k, v, scale, weight):
    """The definition with every key counted weight[t] times, as the kernel returns it."""
    D, keep = q.shape[2], np.repeat(np.arange(len(k)), weight)
    seen = np.ones((len(q), len(keep)), bool)
    o, _, lse, _ = ref.rows_attention(q.double().numpy(), [0, len(q)], [k[keep]], [v[keep]], [seen], scale)
    return torch.from_numpy(o).to(torch.bfloat16), torch.from_numpy(lse).float()


@pytest.mark.parametrize("D,Hq,Hkv,n,lens", CASES)
def test_the_bound_rejects_a_lost_and_a_doubled_group(D, Hq, Hkv, n, lens):
    rng, L, scale = np.random.default_rng(D + n), max(lens), D ** -0.5
    q = torch.from_numpy(rng.standard_normal((1, 1, D)) * 0.5).to(torch.bfloat16)  # the last row, which sees all
    k = torch.from_numpy(rng.standard_normal((L, 1, D))).to(torch.bfloat16).double().numpy()
    v = marks(np.arange(L), D)[:, None]
    want, m = want_of_cpu(q, k, v, L, scale)
    once = np.ones(L, int)
    check(*result(q, k, v, scale, once), want, m, D, "itself")
    for g in sorted({0, 1, L // 32, L // 16 - 2, *rng.integers(0, L // 16, 6).tolist()}):
        for times in (0, 2):
            weight = once.copy()
            weight[16 * g:16 * g + 16] = times
            with pytest.raises(AssertionError):
                check(*result(q, k, v, scale, weight), want, m, D, "cut")


def want_of_cpu(q, k, v, L, scale):
    return want_of(q, [0, 1], [k], [v], [L - 1], None, scale, None)
