"""Bounded waits of the attention of several new rows run out, and the library reports it.

As test_wait_timeout_served_gpu.py, with the wait-test build: a workspace hook word leaves an arrival, a copy or an item out."""
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
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "wait_rows_child.py")], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    from weight_streaming_gb300 import _lib as V
    lines = out.stdout.strip().splitlines()
    assert len(lines) == 61, out.stdout
    for line in lines:
        assert line.endswith(f": {V.VP_OK} {V.VP_ERR_TIMEOUT} {V.VP_OK} 1"), line
