"""What the chunked gated delta rule keeps of its numbers where a norm over
everything does not show it: bf16 outputs, states and gradients behind strong
decays.  The formats' bounds are those of the parity tests."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, err_state, host64
from tests.test_gpu_delta import TOL_SPLIT, cuda, f64, inputs
from tests.test_gpu_delta_backward import TOL

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


@pytest.mark.parametrize("B,N,Hk,H,dk,dv", [
    (1, 70, 1, 1, 64, 24), (1, 130, 2, 4, 128, 64), (1, 100, 1, 1, 256, 40),   # blocks of one group of columns
    (2, 400, 4, 8, 128, 200), (3, 300, 2, 6, 64, 200),                         # of two
    (4, 330, 8, 16, 128, 128), (4, 200, 8, 16, 256, 168), (4, 150, 8, 16, 64, 136),  # of four
])
def test_a_bf16_output_is_the_fp32_one_rounded(B, N, Hk, H, dk, dv):
    f, s0 = inputs(941, B, N, Hk, H, dk, dv, "bf16")
    kw = dict(initial_state=s0.cuda(), want_final_state=True)
    wide, S = R.ret_delta_forward_chunkwise(**cuda(f), out_dtype=torch.float32, **kw)
    out, S16 = R.ret_delta_forward_chunkwise(**cuda(f), out_dtype=torch.bfloat16, **kw)
    assert torch.equal(out, wide.to(torch.bfloat16)) and torch.equal(S, S16)


def behind(f, g, rows):
    """Decays of e^g at ``rows``, a few hundredths elsewhere."""
    f["g"] = f["g"] * 0.05
    f["g"][:, rows] = g


# dinitial_state itself, of its own norm, when all of it passes a decay: of every
# token, of the first one, in a first chunk without a gradient of its own; with and
# without a gradient of the final state.
@pytest.mark.parametrize("final", [False, True])
@pytest.mark.parametrize("N,dk,dv,g,rows,quiet", [
    (1, 64, 40, -10.0, slice(None), 0), (1, 256, 168, -25.0, slice(None), 0), (5, 128, 64, -20.0, slice(None), 0),
    (66, 64, 64, -20.0, slice(None), 0), (130, 64, 72, -18.0, slice(0, 1), 0), (130, 128, 64, -40.0, slice(0, 1), 0),
    (200, 256, 40, -15.0, slice(0, 1), 64), (200, 64, 200, -60.0, slice(0, 1), 100),
])
def test_the_initial_states_gradient_behind_a_strong_decay(N, dk, dv, g, rows, quiet, final):
    B, H = 2, 4
    f, s0 = inputs(942, B, N, H, H, dk, dv, "bf16")
    behind(f, g, rows)
    dout, dS = dev(make_tensor(942, 4, (B, N, H, dv), "bf16")), make_tensor(942, 5, (B, H, dk, dv), "f32", 0.3)
    dout[:, :quiet] = 0
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dout, initial_state=s0.cuda(), dfinal_state=dev(dS) if final else None)
    ref = od.delta_backward(**f64(f), dout=host64(dout), initial_state=host64(s0), dfinal_state=dS.f64 if final else None)
    assert np.abs(ref["dinitial_state"]).max() < 1e-3  # it is small, and not zero
    assert err_state(host64(got[5]), ref["dinitial_state"]) < TOL


# The mirror image: nothing written behind the last tokens' decay.
@pytest.mark.parametrize("N,dk,dv,g,last", [(3, 64, 40, -10.0, 1), (64, 128, 64, -20.0, 1), (66, 256, 72, -15.0, 2), (200, 64, 136, -50.0, 1)])
def test_the_final_state_behind_a_strong_decay(N, dk, dv, g, last):
    B, H = 2, 4
    f, s0 = inputs(943, B, N, H, H, dk, dv, "bf16")
    behind(f, g, slice(N - last, N))
    f["beta"][:, N - last:] = 0
    _, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), want_final_state=True)
    _, ref = od.delta_forward(**f64(f), initial_state=host64(s0))
    assert np.abs(ref).max() < 1e-3
    assert err_state(host64(S), ref) < TOL_SPLIT


# Halves of a state's rows many powers of two apart: finite, and good to 2^-18 of the
# output's norm, whichever half is the larger and whichever the queries read.
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low,high", [(50, -85), (-85, 50), (0, -80), (-60, 60)])
@pytest.mark.parametrize("dk", [64, 256])
def test_halves_of_a_state_far_apart(dk, low, high, out_dtype):
    B, N, H, dv = 1, 70, 2, 40
    f, s0 = inputs(944, B, N, H, H, dk, dv, "bf16")
    s0[:, :, :dk // 2] *= 2.0 ** low
    s0[:, :, dk // 2:] *= 2.0 ** high
    f["beta"].zero_()  # nothing written: a write would spread one half's size over the other
    f["g"].zero_()
    f["q"][:, :20, :, :dk // 2] = 0
    f["q"][:, 20:40, :, dk // 2:] = 0
    out, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out_dtype=out_dtype, want_final_state=True)
    ref, _ = od.delta_forward(**f64(f), initial_state=host64(s0))
    assert torch.equal(S.cpu(), s0) and torch.isfinite(out).all()
    assert np.linalg.norm(host64(out) - ref) <= (TOL_SPLIT if out_dtype == torch.float32 else 2.0 ** -8) * np.linalg.norm(ref)
