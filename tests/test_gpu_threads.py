"""Several host threads use the same handles of the training operators at once, from a process's
first calls on (GPU): each on a stream of its own, and all with one thread's results."""
import os
import subprocess
import sys

import pytest

from _gpu import ensure_built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys, threading
sys.path.insert(0, sys.argv[1])
import torch
import residual_gradient_compression_gb300 as ac

THREADS, rows, dim = 8, 70, 1024
dev = torch.device("cuda", 0)
torch.manual_seed(0)
x, dy = torch.randn(rows, dim, device=dev), torch.randn(rows, dim, device=dev)
w = torch.ones(dim, device=dev)
shapes = [(3, 300, 64), (16, 90, 1024), (2, 2000, 7)]  # clusters, many columns, all chunks at once
seqs = [[torch.randn(s, device=dev) for _ in range(3)] for s in shapes]
norm, recs = ac.adacomp_layer_norm_init(dim), [ac.adacomp_recurrence_init(s[2]) for s in shapes]
torch.cuda.synchronize()
results, errors = [None] * THREADS, []
start = threading.Barrier(THREADS)

def work(i):
    try:
        torch.cuda.set_device(dev)
        with torch.cuda.stream(torch.cuda.Stream()):
            y, dx = torch.empty_like(x), torch.empty_like(x)
            mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
            dw, db = torch.empty_like(w), torch.empty_like(w)
            ws = torch.empty(ac.adacomp_layer_norm_backward_ws_bytes(norm, rows), dtype=torch.uint8, device=dev)
            out = [y, dx, dw, db]
            outs = [[torch.empty_like(z) for _ in range(3)] for z, _, _ in seqs]
            carries = [torch.empty(ac.adacomp_recurrence_carry_bytes(h, s[0], s[1]) // 4, device=dev)
                       for h, s in zip(recs, shapes)]
            start.wait()
            ac.adacomp_layer_norm_forward(norm, x, w, None, y, mean, rstd)
            ac.adacomp_layer_norm_backward(norm, dy, x, w, mean, rstd, dx, dw, db, ws)
            for h, (z, v, g), (o, dz, dv), carry in zip(recs, seqs, outs, carries):
                ac.adacomp_recurrence_forward(h, z, v, o, carry=carry)
                ac.adacomp_recurrence_backward(h, z, v, g, carry, dz, dv)
            torch.cuda.current_stream().synchronize()
            results[i] = out + [t for o in outs for t in o]
    except Exception as e:
        errors.append(repr(e))

threads = [threading.Thread(target=work, args=(i,)) for i in range(THREADS)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not errors, errors
first = results[0]
work_alone = threading.Barrier(1)
start = work_alone
work(0)
for r in results[1:] + [results[0]]:
    assert all(torch.equal(a, b) for a, b in zip(r, first))
print("same")
"""


def test_first_calls_of_several_threads():
    ensure_built()
    r = subprocess.run([sys.executable, "-c", CODE, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
