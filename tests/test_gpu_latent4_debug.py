"""The 4-bit cache's calls in the debug build: results as in the release build,
and a wait of the decode kernel that runs out ends the call in order."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import ctypes
import time
import torch
import kda_linear_attention_gb300 as kda
assert kda.library_path().endswith("libkda_gb300_debug.so"), kda.library_path()
NONE = 0xffffffff
torch.manual_seed(1)


def normal(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


# the first block has eight tiles of positions, of two sequences, in its units
N, L, page = 200, 700, 64
per = -(-L // page)
table = torch.randperm(N * per, device="cuda").to(torch.int32).view(N, per)
lens = torch.full((N,), L, dtype=torch.int32, device="cuda")
cu = torch.arange(0, N * L + 1, L, dtype=torch.int32, device="cuda")
turns, _ = kda.rotary_turns()
cache = torch.zeros((N * per, page, 416), dtype=torch.uint8, device="cuda")
kda.latent4_append(normal(N * L, 576), cache, table, lens, cu, turns=turns)
drop = kda.lib().kda_debug_latent4_leave_out
drop.argtypes = [ctypes.c_uint]
for heads in (5, 48, 64):
    q = normal(N, heads, 576)
    kda.latent_rotate(q[..., 512:], turns, lens)
    call = lambda: kda.latent4_decode(q, cache, table, lens)
    kda.device_error(reset=True)
    want = call()
    torch.cuda.synchronize()
    assert kda.device_error(reset=True) == 0
    for tile in (0, 1, 3, 4, 5, 7) if heads == 5 else (2, 5):
        assert drop(tile) == 0
        start = time.time()
        call()
        torch.cuda.synchronize()
        took = time.time() - start
        assert drop(NONE) == 0
        assert kda.device_error(reset=True) == 1, (heads, tile)
        assert took < 20, (heads, tile, took)
        for _ in range(2):
            got = call()
            torch.cuda.synchronize()
            assert kda.device_error(reset=True) == 0
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (heads, tile)
        print(heads, tile, "%.2f s" % took)
print("waits ran out in order")
'''


def test_decode4_waits_that_run_out_end_in_order():
    """One softmax warp leaves out its arrival, so the wait for it runs out (the
    debug build's limit is a second): the call ends, the error word says so, and
    the calls after it are right."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_linear_attention_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, KDA_GB300_DEBUG="1", PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "waits ran out in order" in r.stdout
