"""Python's garbage collector beside captures: GPU tests run with it on and start without what earlier ones left, and a chain
that it destroys in a capture does not end that capture."""

import gc
import os
import subprocess
import sys
import weakref

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LEFT = []


class _Ring:
    def __init__(self):
        self.self = self
        self.graph = torch.cuda.CUDAGraph()


def test_collector_is_on():
    assert gc.isenabled()


@pytest.mark.parametrize("generation", [0, 1, 2])
def test_ring_left_behind(generation):
    """A graph that only the collector can free, in each of its generations; looked for by the test after this one."""
    LEFT.append(weakref.ref(_Ring()))
    for g in range(generation):
        keep = LEFT[-1]()
        gc.collect(g)
        del keep


def test_ring_is_gone():
    assert len(LEFT) == 3 and all(r() is None for r in LEFT)


CAPTURE = r"""
import gc, os, sys, torch
import tile_level_sync_gb300 as cs
status = 1
try:
    x = torch.zeros(64, device="cuda")
    chain = cs.Chain(cs.make_desc(cs.CHAIN_MLP_GELU, "ROW", M=64, K=256, N1=256, N2=256, flags=cs.FLAG_TRACE))
    ring = [chain]
    ring.append(ring)
    left = cs.Chain(cs.make_desc(cs.CHAIN_MLP_GELU, "STREAM", M=64, K=256, N1=256, N2=256))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x += 1
        del chain, ring
        gc.collect()
        x += 2
        left.close()
        x += 4
    g.replay()
    torch.cuda.synchronize()
    status = 0 if bool((x == 7).all()) else 2
    print("sum", float(x[0]), flush=True)
except BaseException as e:
    print(type(e).__name__, e, flush=True)
os._exit(status)  # a capture that was ended takes the process with it at its exit
"""


def test_chains_destroyed_in_a_capture():
    r = subprocess.run([sys.executable, "-c", CAPTURE], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "sum 7.0" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]
