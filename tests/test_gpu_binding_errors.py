"""Errors of the entry points that the direct binding calls: raised, with nothing
done twice and nothing left for the next call."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def step(off=0):
    """A decode step's arguments; q starts ``off`` elements behind an aligned address."""
    B, H, d = 2, 2, 64
    flat = torch.randn(B * H * d + 8, device="cuda").bfloat16()
    q = flat[off:off + B * H * d].view(B, H, d)
    return (q, q.clone() / 8, torch.randn(B, H, d, device="cuda").bfloat16(), -torch.rand(B, H, device="cuda"),
            torch.rand(B, H, device="cuda"), torch.randn(B, H, d, d, device="cuda"))


def test_a_refusal_is_a_status_and_raised():
    a = step(1)
    before = a[5].clone()
    assert R._binding.delta_decode_step(*a, False) == R.RET_ERR_INVALID_ARG
    with pytest.raises(R.RetentionError, match="16-byte aligned"):
        R.ret_delta_decode_step(*a)
    assert torch.equal(a[5], before)


def test_an_earlier_error_is_not_the_next_launchs():
    """A call that CUDA refuses on the host (a synchronisation while its stream is
    captured) reports its error; the decode step after it is one step and no error."""
    script = """
import torch
import linear_recurrent_sequence_chunkwise_b200 as R
from tests.test_gpu_binding_errors import step
import tests.test_gpu_binding_errors as t
t.R = R
a = step()
S = a[5].clone()
want = R.ret_delta_decode_step(*a[:5], S)
torch.cuda.synchronize()
s = torch.cuda.Stream()
graph = torch.cuda.CUDAGraph()
with torch.cuda.stream(s):
    graph.capture_begin()
    try:
        R.ret_check_device_error()
        raise SystemExit("not refused")
    except R.RetentionError as e:
        assert e.status == R.RET_ERR_CUDA, e
    try:
        graph.capture_end()
    except RuntimeError:
        pass  # the capture is lost, and says so
S2 = a[5].clone()
got = R.ret_delta_decode_step(*a[:5], S2)
torch.cuda.synchronize()
assert torch.equal(got, want) and torch.equal(S2, S)
print("one step")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", script], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "one step" in r.stdout, r.stdout + r.stderr
