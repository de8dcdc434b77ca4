"""Child process of test_wait_timeout_served_gpu.py (run with VP_LIBVERIFY naming the wait-test build of the
library, whose bounded waits give up after milliseconds).

Each case runs normally; then the workspace's test hook leaves an arrival or a copy out, or gives a wait
up, so that a wait of the kernel runs out: the call must return and the status word read VP_ERR_TIMEOUT;
then, after vp_workspace_init, the next call must give the first one's results.  Prints "case: status status
status equal" per case."""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from helpers import workspace  # noqa: E402
from test_served_layer_gpu import Paged, bf16, i32  # noqa: E402
from weight_streaming_gb300 import _lib as V  # noqa: E402

HOOK_WORD = 32 // 4  # int32 index of the hook word (byte offset 32 from the status word)


def attention(S, Hq, Hkv, D, P, n):
    rng = np.random.default_rng(S + D)
    p = Paged(V, 1, S, -(-n // P), P, Hkv, D)
    q, lens = bf16(rng, (S, Hq, D), 1.5), i32([n] * S)
    out, lse = torch.zeros((S, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((S, Hq), device="cuda")
    ws = workspace(V.vp_paged_attention_workspace_bytes(S, Hq, Hkv, D))

    def run():
        V.vp_paged_attention(p.desc(), q, lens, S, Hq, D ** -0.5, None, out, lse, ws)
        torch.cuda.synchronize()
        return out.clone(), lse.clone()
    return run, ws


def linear(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    kb, nb = -(-K // 128), -(-N // 128)
    xq, wq = (torch.randint(0, 120, s, generator=g, device="cuda").to(torch.uint8) for s in ((M, K), (N, K)))
    xs, wsc = torch.rand((M, kb), generator=g, device="cuda"), torch.rand((nb, kb), generator=g, device="cuda")
    packed = torch.empty(V.vp_packed_bytes_fp8_block(N, K), dtype=torch.uint8, device="cuda")
    V.vp_pack_fp8_block(wq, N, K, packed)
    y = torch.zeros((M, N), device="cuda")
    ws = workspace(V.vp_linear_fp8_block_workspace_bytes(M, N, K))

    def run():
        V.vp_linear_fp8_block(packed, wsc, xq, xs, y, V.VP_F32, M, N, K, ws)
        torch.cuda.synchronize()
        return (y.clone(),)
    return run, ws


LINEAR = {
    "parts in a cluster": (8, 5120, 17408),
    "parts in a cluster, 32 columns": (24, 5120, 17408),
    "parts in the workspace": (60, 5120, 17408),
    "tokens on the lanes": (100, 5120, 17408),
    "more tiles than CTAs": (8, 19600, 5136),
    "pairs": (200, 16384, 5120),
    "pairs, whole rounds and parts": (1024, 5120, 5120),
}
ATTENTION = {
    "one long sequence": (1, 6, 1, 256, 64, 16 * 152 * 20),
    "a group of 16": (1, 16, 1, 128, 16, 32 * 152 * 18),
    "whole sequences": (400, 6, 1, 256, 64, 400),
    "runs over their borders": (60, 8, 2, 128, 32, 3000),
}


def main():
    assert "waittest" in V.LIB_PATH, V.LIB_PATH
    cases = [(f"attention, {name}, hook {h}", attention, shape, h) for name, shape in ATTENTION.items()
             for h in ((1, 2, 4) if name == "whole sequences" else (1, 2, 3, 4))]
    cases += [(f"linear, {name}, hook {h}", linear, shape, h) for name, shape in LINEAR.items()
              for h in ((1, 2, 3, 4, 5, 6) if "pairs" in name else (1, 2, 3, 4, 6))]
    for what, make, shape, hook in cases:
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
        print(f"{what}: {st[0]} {st[1]} {st[2]} {int(equal)}", flush=True)


if __name__ == "__main__":
    main()
