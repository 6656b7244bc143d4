"""The example that runs the losses and the shard step together: the student
learns what the teacher recorded. It runs as a user runs it, in a process of
its own (its matrix products keep a workspace in the allocator of theirs)."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_distill_example_learns():
    p = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "distill.py"), "40"],
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stdout + p.stderr
    losses = [float(x) for x in re.findall(r"distillation loss (-?[0-9.]+)", p.stdout)]
    held_out = [float(x) for x in re.findall(r"log probability (-?[0-9.]+)", p.stdout)]
    assert len(losses) == 5 and losses[-1] < 0.8 * losses[0], p.stdout
    assert len(held_out) == 2 and held_out[1] > held_out[0] + 0.3, p.stdout
