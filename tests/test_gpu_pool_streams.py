"""The compute/copy stream pair in a process that has made and destroyed streams before: the two stay on hardware
queues of their own. Streams keep their queue for a process's life, so each case is a process of its own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes as C, sys, time
import torch
from nf4_weight_streamed_amd import lib

made, gone = int(sys.argv[1]), [int(i) for i in sys.argv[2].split(",") if i]
a, b = (torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16) for _ in range(2))
c = torch.empty_like(a)
hip = C.CDLL("libamdhip64.so.7")                    # the process's own runtime
streams = [C.c_void_p() for _ in range(made)]
for s in streams:
    assert hip.hipStreamCreateWithFlags(C.byref(s), C.c_uint(1)) == 0     # non-blocking, default priority
for i in gone:
    assert hip.hipStreamDestroy(streams[i]) == 0
comp, copy = lib.pool_streams()
nb, nbytes = 8, 128 << 20
host = lib.pinned_empty(nb * nbytes)
slab = torch.empty(2 * nbytes, dtype=torch.uint8, device="cuda")
pool = lib.StreamPool([host[i * nbytes:(i + 1) * nbytes] for i in range(nb)], slab, nbytes, 2, copy)

def one_pass(copies, compute):
    with torch.cuda.stream(comp):
        for i in range(nb):
            if copies:
                pool.acquire(i)
                if i + 1 < nb:
                    pool.prefetch(i + 1)
            for _ in range(2 if compute else 0):
                torch.matmul(a, b, out=c)
            if copies:
                pool.release(i)

def timed(*args):
    best = float("inf")
    for _ in range(3):
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        one_pass(*args)
        torch.cuda.synchronize()
        best = min(best, time.perf_counter() - t0)
    return best

one_pass(True, True)
print(*(timed(*args) for args in ((True, False), (False, True), (True, True))), flush=True)
pool.close()
"""


# streams made, and which of them are destroyed: a queue of four (every fourth stream) left short by three, two left
# short by two, and nothing left
@pytest.mark.parametrize("made,gone", [(12, [0, 4, 8]), (12, [1, 5, 9]), (12, [2, 6, 10]), (12, [3, 7, 11]),
                                       (10, [0, 1, 4, 5]), (5, [0, 1, 2, 3, 4])])
def test_pair_overlaps_after_streams_were_destroyed(gpu_lib, made, gone):
    r = subprocess.run([sys.executable, "-c", CHILD, str(made), ",".join(map(str, gone))], cwd=ROOT, capture_output=True,
                       text=True, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    copies, compute, both = (float(x) for x in r.stdout.split())
    print(f"copies {copies * 1e3:.2f} ms, compute {compute * 1e3:.2f} ms, both {both * 1e3:.2f} ms", flush=True)
    assert compute > 0.3 * copies, "the compute must be long enough for the check to mean something"
    # on one queue they would run one after the other
    assert both < copies + 0.5 * compute, (copies, compute, both)
