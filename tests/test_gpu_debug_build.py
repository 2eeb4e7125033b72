"""The debug build (python -m kda_linear_attention_gb300.build --debug,
selected with KDA_GB300_DEBUG=1): the same kernels with index checks on
their global-memory addressing, standing in for a memory checker.  On valid
inputs no check may fire and the results must keep parity with the oracle;
run in a child process so that the debug library is the one loaded."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r'''
import numpy as np, torch
import kda_inputs as ki, oracle
from oracle import layer as olayer
import kda_linear_attention_gb300 as kda
from kda_testlib import TOL_BF16, TOL_F32, assert_close, dev_tensor, prefill_on_gpu, decode_on_gpu
assert kda.library_path().endswith("libkda_gb300_debug.so"), kda.library_path()
kda.device_error(reset=True)
for dtype, chunk in (("bf16", 64), ("bf16", 32), ("f32", 16)):
    inp = ki.gen_prefill(901, [0, 1, 17, 64, 65, 200], H=3, dtype=dtype, chunk=chunk, with_s0=True)
    o, S = prefill_on_gpu(inp)               # asserts a clear error word
    o_ref, S_ref = oracle.prefill(inp)
    tol = TOL_F32 if dtype == "f32" else TOL_BF16
    assert_close(o, o_ref, tol, "debug prefill o %s/%d" % (dtype, chunk))
    assert_close(S, S_ref, tol, "debug prefill S %s/%d" % (dtype, chunk))
rng = np.random.Generator(np.random.PCG64(902))
S0 = ki.gen_decode_state(rng, 5, 4)
step = ki.gen_decode_step(rng, 5, 4, "bf16")
Sd = dev_tensor(S0)
od = decode_on_gpu(Sd, step)
o_ref, S_ref = oracle.decode(S0, step)
assert_close(od, o_ref, TOL_BF16, "debug decode o")
idx = np.array([3, -1, 0, 4, 1], dtype=np.int32)
d = {n: dev_tensor(getattr(step, n)) for n in ("q", "k", "v", "g", "beta")}
pool = dev_tensor(ki.gen_decode_state(rng, 6, 4))
kda.decode_step_pool(d["q"], d["k"], d["v"], d["g"], d["beta"], pool, state_indices=dev_tensor(idx))
L = ki.gen_layer(903, [0, 3, 64, 130], H=2, with_conv0=True)
q, k, v, co = kda.conv_prologue(dev_tensor(L.xq), dev_tensor(L.xk), dev_tensor(L.xv), dev_tensor(L.conv_w),
                                dev_tensor(L.cu_seqlens), conv_in=dev_tensor(L.conv0).view(torch.bfloat16))
torch.cuda.synchronize()
err = kda.device_error(reset=True)
assert err == 0, "a debug index check fired on valid inputs: 0x%x" % err
print("debug build clean")
'''


def test_debug_build_is_clean_on_valid_inputs():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_linear_attention_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, KDA_GB300_DEBUG="1",
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests"), os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug build clean" in r.stdout


WAITS = r'''
import time
import numpy as np, torch
import kda_linear_attention_gb300 as kda
assert kda.library_path().endswith("libkda_gb300_debug.so"), kda.library_path()
NONE = 0xffffffff
torch.manual_seed(1)


def normal(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def run(name, call, drop):
    kda.device_error(reset=True)
    want = call()
    torch.cuda.synchronize()
    assert kda.device_error(reset=True) == 0
    for tile in (0, 1, 3, 4, 5, 7):
        assert drop(tile) == 0
        start = time.time()
        call()
        torch.cuda.synchronize()
        took = time.time() - start
        assert drop(NONE) == 0
        assert kda.device_error(reset=True) == 1, (name, tile)
        assert took < 20, (name, tile, took)
        for _ in range(2):
            got = call()
            torch.cuda.synchronize()
            assert kda.device_error(reset=True) == 0
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (name, tile)
        print(name, tile, "%.2f s" % took)


# the first block has eight tiles of positions, of two sequences, in its units
N, L, page = 200, 700, 64
per = -(-L // page)
cache, q = normal(N * per, page, 576), normal(N, 5, 576)
table = torch.randperm(N * per, device="cuda").to(torch.int32).view(N, per)
lens = torch.full((N,), L, dtype=torch.int32, device="cuda")
drop = kda.lib().kda_debug_latent_leave_out
drop.argtypes = [__import__("ctypes").c_uint] * 2
run("decode", lambda: kda.latent_decode(q, cache, table, lens), lambda t: drop(t, NONE))
# 320 work tiles of one to ten key tiles: the first block takes over further ones
T, H = 1300, 64
cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
pq, kv, pe = normal(T, H, 192), normal(T, H, 256), normal(T, 64)
run("prefill", lambda: kda.latent_prefill(pq, kv, pe, cu), lambda t: drop(NONE, t))
print("waits ran out in order")
'''


def test_latent_waits_that_run_out_end_in_order():
    """One softmax warp leaves out its arrival, so the product warp's wait runs
    out (the debug build's limit is a second): the call ends, the error word
    says so, and the calls after it are right."""
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from kda_linear_attention_gb300 import build
    build.build(debug=True)
    env = dict(os.environ, KDA_GB300_DEBUG="1", PYTHONPATH=os.pathsep.join([ROOT, os.environ.get("PYTHONPATH", "")]))
    r = subprocess.run([sys.executable, "-c", WAITS], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "waits ran out in order" in r.stdout
