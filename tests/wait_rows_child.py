"""Child process of test_wait_timeout_rows_gpu.py (run with VP_LIBVERIFY naming the wait-test build of the library, whose
bounded waits give up after milliseconds): as wait_served_child.py, for the attention of several new rows per sequence.

Prints "case: status status status equal" per case."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from helpers import workspace  # noqa: E402
from test_rows_attention_gpu import Cache  # noqa: E402
from test_served_layer_gpu import bf16, i32  # noqa: E402
from weight_streaming_gb300 import _lib as V  # noqa: E402

HOOK_WORD = 32 // 4  # int32 index of the hook word (byte offset 32 from the status word)


def prompt(D, Hq, Hkv, n):
    q, kv = bf16(np.random.default_rng(n), (n, Hq, D)), bf16(np.random.default_rng(D), (n, 2 * Hkv, D))
    ws = workspace(V.vp_prompt_attention_workspace_bytes(1, n, Hq, Hkv, D))
    out, lse, ld, start = torch.zeros_like(q), torch.zeros((n, Hq), device="cuda"), 2 * Hkv * D, i32([0, n])

    def run():
        V.vp_prompt_attention(q, Hq * D, kv, ld, kv[:, Hkv:], ld, start, 1, n, Hq, Hkv, D, D ** -0.5, None, out, lse, ws)
        torch.cuda.synchronize()
        return out.clone(), lse.clone()
    return run, ws


def rows(fp8, D, Hq, Hkv, S, n, L):
    c, M = Cache(V, 1, S, -(-L // 32), 32, Hkv, D, fp8), S * n
    q = bf16(np.random.default_rng(n), (M, Hq, D))
    ws = workspace(V.vp_paged_attention_rows_workspace_bytes(S, M, Hq, Hkv, D))
    out, lse, start, lens = torch.zeros_like(q), torch.zeros((M, Hq), device="cuda"), i32(np.arange(S + 1) * n), i32([L] * S)

    def run():
        c.attend(q, start, lens, M, Hq, D ** -0.5, None, out, lse, ws)
        torch.cuda.synchronize()
        return out.clone(), lse.clone()
    return run, ws


CASES = [(f"prompt {s}", prompt, s) for s in ((128, 8, 2, 1500), (64, 4, 2, 900), (256, 6, 1, 1200))]
CASES += [(f"rows {s}", rows, s) for s in ((False, 128, 4, 1, 20, 1, 77), (False, 256, 8, 1, 3, 6, 100), (False, 256, 4, 2, 2, 200, 401),
                                           (True, 128, 4, 1, 20, 1, 77), (True, 256, 8, 1, 3, 6, 333), (True, 128, 8, 2, 2, 200, 401),
                                           (True, 256, 6, 1, 2, 100, 9000), (True, 64, 2, 1, 30, 1, 700))]


def main():
    assert "waittest" in V.LIB_PATH, V.LIB_PATH
    for what, make, shape in CASES:
        pair = 256 in shape and shape[-1] in (1200, 401, 9000)
        for hook in (1, 2, 3, 4, 5, 6, 7) if pair else (1, 2, 3, 4, 5):
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
