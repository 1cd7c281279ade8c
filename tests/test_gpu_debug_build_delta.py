"""The delta rule and the gradients of the debug library (KATA_DEBUG=1): each entry point on
tiny shapes against its definition in 64 bits, with a clean status (GPU). In a child
process, which loads libkata_debug.so in place of libkata.so."""
import os
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parent.parent

SCRIPT = r'''
import sys
sys.path.insert(0, ROOT); sys.path.insert(0, ROOT + "/tests")
import torch
import kernelized_linear_attention_chunked_b200 as kata
from _delta_ref import delta_forward, delta_grads, delta_inputs, prefill_grads, rel

assert kata.debug_build()
names = ("q", "k", "v", "g", "beta")
for dtype in (torch.float32, torch.bfloat16):
    tol = 2e-5 if dtype == torch.float32 else 6e-3
    for d in (16, 32, 64, 128):
        x = delta_inputs(1, 2, 70, d, dtype, seed=d)
        seq = [x[n] for n in names]
        o, S = kata.delta_prefill(*seq, S_in=x["S"])
        kata.sync_status()
        ro, rS = delta_forward(*seq, d ** -0.5, x["S"])
        assert rel(o, ro) < tol and rel(S, rS) < 2e-5
        got = kata.delta_backward(*seq, x["do"], S_in=x["S"], dS=x["dS"], state_grad=True)
        kata.sync_status()
        for a, b in zip(got, delta_grads(*seq, d ** -0.5, x["do"], x["S"], x["dS"])):
            assert rel(a, b) < (tol if a.dtype == dtype else 2e-5)
        S = x["S"].clone()
        o = kata.delta_decode_step(*(t[:, :, 0].contiguous() for t in seq), S)
        kata.sync_status()
        ro, rS = delta_forward(*(t[:, :, :1] for t in seq), d ** -0.5, x["S"])
        assert rel(o, ro[:, :, 0]) < tol and rel(S, rS) < 2e-5
        if d < 128:
            y = (x["q"], x["k"], x["v"], x["do"])
            got = kata.prefill_backward(*y)
            kata.sync_status()
            for a, b in zip(got, prefill_grads(*y, 1e-6)):
                assert rel(a, b) < tol
print("CLEAN")
'''


def test_entry_points_run_clean():
    code = f"ROOT = {str(ROOT)!r}\n" + SCRIPT
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, KATA_DEBUG="1"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "CLEAN" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
