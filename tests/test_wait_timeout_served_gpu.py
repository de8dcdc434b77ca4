"""Bounded waits of the served attention layer's kernels run out, and the library reports it.

As test_wait_timeout_gpu.py, with the wait-test build: a workspace hook word leaves an arrival or a copy out, or gives a wait up."""
import importlib
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_waits_that_run_out_are_reported_and_leave_nothing_behind():
    build = importlib.import_module("weight_streaming_gb300.build")
    env = dict(os.environ, VP_LIBVERIFY=build.build(variant="waittest"))
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "wait_served_child.py")], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    from weight_streaming_gb300 import _lib as V
    lines = out.stdout.strip().splitlines()
    assert len(lines) == 52, out.stdout
    for line in lines:
        assert line.endswith(f": {V.VP_OK} {V.VP_ERR_TIMEOUT} {V.VP_OK} 1"), line
