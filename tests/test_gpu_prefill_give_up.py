"""Prefill when waits run out: the kernel flags it and ends, whichever warps gave up, and the next call on
the same workspace is right. In a process of its own, with the build that has this switch."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_warps_that_give_up_leave_together():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    script = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_give_up.py")
    r = subprocess.run([sys.executable, script], capture_output=True, text=True, timeout=300)
    print(r.stdout, r.stderr)
    assert r.returncode == 0
    lines = r.stdout.strip().splitlines()
    assert len(lines) == 8
    for line in lines:
        flags, seconds, after, _ = line.split(": ")[1].split()
        assert int(flags) == 0x8 and int(after) == 0 and float(seconds) < 10
