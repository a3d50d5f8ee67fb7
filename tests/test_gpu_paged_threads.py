"""Paged batches from several host threads at once, each with its own stream and workspace, from
the first call of the process's libraries on: results, launch counts and error messages are each
thread's own."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = """
import sys
sys.path[:0] = ["tests", "."]
import threading

import torch
import top_kv_routing_b200 as msa
from paged_ref import Batch

CASES = [dict(new=[1] * 40, past=[25] * 40, L=4, H=16, G=4, groups=[0, 40], mem=[900]),
         dict(new=[50] * 6, past=[40] * 6, L=4, H=16, G=4, groups=[0, 6], mem=[500]),
         dict(new=[1] * 9, past=[700] * 9, L=2, H=4, G=4),
         dict(new=[5] * 7, past=[0, 1, 11, 12, 100, 250, 31], L=2, H=2, G=4, groups=[0, 7], mem=[200])]
LAUNCHES = [2, 1, 1, 1]
xs = [Batch(seed=81 + i, **c) for i, c in enumerate(CASES)]
for x in xs:
    n = msa.msa_shared_attend_workspace_size(x.T, x.B, x.NG, x.L, x.HQ, x.H)
    x.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    x.q_rot = torch.empty_like(x.out)
torch.cuda.synchronize()
streams = [torch.cuda.Stream() for _ in xs]
start, failed = threading.Barrier(len(xs)), []


def work(i):
    x, s = xs[i], streams[i]
    try:
        start.wait()
        for _ in range(200):
            assert x.call_append(msa, q_rot=x.q_rot, stream=s) == 1
            x.q_plain, x.q = x.q, x.q_rot
            assert x.call_attend(msa, stream=s) == LAUNCHES[i]
            x.q = x.q_plain
            try:
                x.call_attend(msa, stream=s, scale=-1.0 - i)
                raise AssertionError("not refused")
            except msa.MsaError as e:
                assert "softmax_scale" in str(e)
    except BaseException as e:
        failed.append((i, repr(e)))


threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not failed, failed
for x in xs:
    x.q = x.q_rot
    x.check()
    assert x.err.item() == 0
print("done")
"""


def test_threads_at_once_from_the_first_call_on():
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "done" in r.stdout, r.stdout + r.stderr
