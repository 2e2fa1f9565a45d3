"""First launches of several host threads in a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import threading
import torch
from tests.gpu_harness import K
from tests.test_gpu_cross import Case

kvq = K()
cases = [Case(m, 128, 8, 2, [300, 77], [4, 40], seed=m) for m in (0, 1, 2, 3, 4)]
steps = [Case(m, 128, 8, 2, [300, 77], [1, 1], seed=9 + m) for m in (0, 3)]
jobs = cases + steps
works = [torch.zeros(1 << 24, dtype=torch.uint8, device="cuda") for _ in jobs]
streams = [torch.cuda.Stream() for _ in jobs]
torch.cuda.synchronize()
barrier, failed = threading.Barrier(len(jobs)), []

def first(i):
    try:
        barrier.wait()
        jobs[i].run(step=jobs[i] in steps, work=works[i], stream=streams[i])
    except Exception as e:
        failed.append(repr(e))

threads = [threading.Thread(target=first, args=(i,)) for i in range(len(jobs))]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not failed, failed
for c in jobs:
    c.check()
print("every thread launched")
"""


def test_threads_whose_first_calls_meet():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "every thread launched" in r.stdout, r.stderr[-2000:]
