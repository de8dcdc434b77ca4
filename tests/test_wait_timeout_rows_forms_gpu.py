"""Bounded waits run out in the forms of the attention of several new rows that test_wait_timeout_rows_gpu.py leaves out: with both,
all 18 (64, 128, 256 columns; one and two tiles; no cache, a bf16 and an 8-bit one)."""
import importlib
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_waits_that_run_out_in_the_other_forms():
    build = importlib.import_module("weight_streaming_gb300.build")
    env = dict(os.environ, VP_LIBVERIFY=build.build(variant="waittest"))
    out = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "wait_rows_forms_child.py")], cwd=ROOT, env=env,
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0, out.stdout[-2000:] + out.stderr[-3000:]
    from weight_streaming_gb300 import _lib as V
    lines = out.stdout.strip().splitlines()
    assert len(lines) == 40, out.stdout
    for line in lines:
        assert line.endswith(f": {V.VP_OK} {V.VP_ERR_TIMEOUT} {V.VP_OK} 1"), line
