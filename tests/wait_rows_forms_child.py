"""Child process of test_wait_timeout_rows_forms_gpu.py: as wait_rows_child.py, for the forms of the kernel that its cases leave out."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from helpers import workspace  # noqa: E402
from test_served_layer_gpu import bf16, i32  # noqa: E402
from wait_rows_child import HOOK_WORD, rows  # noqa: E402
from weight_streaming_gb300 import _lib as V  # noqa: E402


def prompts(D, Hq, Hkv, S, n):
    M = S * n
    q, kv = bf16(np.random.default_rng(n), (M, Hq, D)), bf16(np.random.default_rng(D), (M, 2 * Hkv, D))
    ws = workspace(V.vp_prompt_attention_workspace_bytes(S, M, Hq, Hkv, D))
    out, lse, ld, start = torch.zeros_like(q), torch.zeros((M, Hq), device="cuda"), 2 * Hkv * D, i32(np.arange(S + 1) * n)

    def run():
        V.vp_prompt_attention(q, Hq * D, kv, ld, kv[:, Hkv:], ld, start, S, M, Hq, Hkv, D, D ** -0.5, None, out, lse, ws)
        torch.cuda.synchronize()
        return out.clone(), lse.clone()
    return run, ws


# (Without codes the preparing warps have work, and hook 4 something to leave out, where the first CTA's part holds an edge block: of
# 700 positions it would hold blocks 0 to 2, and block 5 is the edge.)  One tile without a cache; over the bf16 cache 64 columns in one and two tiles, 128 in two; over the 8-bit one 64 in two
CASES = [(f"prompts {s}", prompts, s) for s in ((64, 2, 1, 20, 40), (128, 4, 1, 20, 30), (256, 8, 2, 10, 16), (128, 16, 1, 9, 2))]
CASES += [(f"rows {s}", rows, s) for s in ((False, 64, 2, 1, 30, 1, 77), (False, 64, 4, 1, 2, 200, 401), (False, 128, 8, 2, 2, 200, 401),
                                           (True, 64, 4, 1, 2, 200, 401))]


def main():
    assert "waittest" in V.LIB_PATH, V.LIB_PATH
    for what, make, shape in CASES:
        for hook in (1, 2, 3, 4, 5):
            run, ws = make(*shape)
            want = run()
            st = [V.vp_read_status(ws)]
            ws.view(torch.int32)[HOOK_WORD] = hook
            torch.cuda.synchronize()
            run()
            st.append(V.vp_read_status(ws))
            V.vp_workspace_init(ws)
            torch.cuda.synchronize()
            got = run()
            st.append(V.vp_read_status(ws))
            equal = all(torch.equal(a, b) for a, b in zip(want, got))
            print(f"{what}, hook {hook}: {st[0]} {st[1]} {st[2]} {int(equal)}", flush=True)


if __name__ == "__main__":
    main()
