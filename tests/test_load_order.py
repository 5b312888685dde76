"""The library and torch share one HIP runtime, whichever is loaded first: a
second copy in the process would be handed the first one's streams and
pointers, and crash."""
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("order", ["g.load(); import torch", "import torch; g.load()"])
def test_one_hip_runtime(order):
    code = ("import gru_recurrence_amd as g\n%s\n"
            "maps = {l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}\n"
            "print(len(maps), sorted(maps))" % order.replace("; ", "\n"))
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("1 "), r.stdout
