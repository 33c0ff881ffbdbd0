"""NaN in rows of the gated delta rule that count.  What the token-by-token
definition makes NaN is NaN; a finite value is the definition's; chunks of 64
tokens before the row, and other heads, are untouched.  (Within its chunk a NaN may
reach rows before it.)"""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, host64
from tests.test_gpu_delta import TOL_F32, TOL_SPLIT, cuda, f64, inputs

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


def agrees(got, ref, tol, name):
    """NaN where the reference is; the rest within tol of the reference's norm."""
    got = host64(got)
    assert not np.isfinite(got[~np.isfinite(ref)]).any(), name
    ok = np.isfinite(got)
    assert np.linalg.norm(got[ok] - ref[ok]) <= tol * np.linalg.norm(ref[ok]) + 1e-30, name


@pytest.mark.parametrize("where", ["g", "beta", "q", "k", "v"])
@pytest.mark.parametrize("dtype,dk,dv", [("bf16", 64, 40), ("bf16", 256, 72), ("f32", 64, 40)])
def test_nan_in_a_row_that_counts(where, dtype, dk, dv):
    B, N, H, t = 1, 200, 2, 70
    f, s0 = inputs(951, B, N, H, H, dk, dv, dtype)
    clean, _ = od.delta_forward(**f64(f), initial_state=host64(s0))
    row = f[where][0, t, 0]
    if where in ("g", "beta"):
        f[where][0, t, 0] = float("nan")
    else:
        row[3] = float("nan")
    tol = TOL_SPLIT if dtype == "bf16" else TOL_F32
    ref, Sref = od.delta_forward(**f64(f), initial_state=host64(s0))
    out, S = R.ret_delta_forward_chunkwise(**cuda(f), initial_state=s0.cuda(), out_dtype=torch.float32, want_final_state=True)
    assert np.isnan(ref[0, t, 0]).any()
    agrees(out, ref, tol, "out")
    agrees(S, Sref, tol, "state")
    assert torch.isfinite(out[0, :64, 0]).all() and torch.isfinite(out[0, :, 1]).all() and torch.isfinite(S[0, 1]).all()
    assert np.linalg.norm(host64(out)[0, :64] - clean[0, :64]) < tol * np.linalg.norm(clean[0, :64])


@pytest.mark.parametrize("where", ["g", "beta", "q", "k", "v", "dout"])
@pytest.mark.parametrize("dk,dv", [(64, 40), (128, 72)])
def test_nan_and_the_gradients(where, dk, dv):
    B, N, H, t = 1, 200, 2, 70
    f, s0 = inputs(952, B, N, H, H, dk, dv, "bf16")
    dout = dev(make_tensor(952, 4, (B, N, H, dv), "bf16"))
    if where in ("g", "beta"):
        f[where][0, t, 0] = float("nan")
    else:
        (dout if where == "dout" else f[where])[0, t, 0, 3] = float("nan")
    ref = od.delta_backward(**f64(f), dout=host64(dout), initial_state=host64(s0))
    got = R.ret_delta_backward_chunkwise(**cuda(f), dout=dout, initial_state=s0.cuda())
    for x, name in zip(got, ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state")):
        agrees(x, ref[name], 2.0 ** -15, name)  # sums of the rows that are left: four kinds of paths, 2^-17 each
        assert torch.isfinite(x[:, 1] if name == "dinitial_state" else x[:, :, 1]).all(), name
