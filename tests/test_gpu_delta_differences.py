"""The gated delta rule's gradients against differences of the GPU's own forward.

Each input moves by its last place (bf16; 2^-8 of itself for the gates and the
state) along the sign of its gradient, both ways: x + d and x - d are exact.  The
forward gives L = <out, dout> + <S, dS> at both, and the difference is <grad, 2 d>
up to the third-order term, which the oracle's own differences and gradients give.

Tolerance: a result of the forward is good to 2^-18 of its norm, so L to 2^-18
(|out| |dout| + |S| |dS|), twice; a gradient to 2^-17 of its norm (dg: of the row
products that it sums)."""
import numpy as np
import pytest
import torch

from oracle import delta as od
from retention_inputs import make_tensor
from tests.helpers import dev, host64
from tests.test_gpu_delta import cuda, f64, inputs

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


NAMES = ("q", "k", "v", "g", "beta", "initial_state")


@pytest.mark.parametrize("B,N,Hk,H,dk,dv", [(1, 100, 1, 2, 64, 64), (2, 70, 1, 1, 128, 40), (1, 130, 2, 2, 256, 24)])
def test_differences_of_the_forward(B, N, Hk, H, dk, dv):
    f, s0 = inputs(971, B, N, Hk, H, dk, dv, "bf16")
    dout, dS = make_tensor(971, 4, (B, N, H, dv), "bf16"), make_tensor(971, 5, (B, H, dk, dv), "f32", 0.3)
    grads = R.ret_delta_backward_chunkwise(**cuda(f), dout=dev(dout), initial_state=s0.cuda(), dfinal_state=dev(dS))
    grads = dict(zip(NAMES, (host64(x) for x in grads)))
    base = {**f, "initial_state": s0}
    ref = od.delta_backward(**f64(f), dout=dout.f64, initial_state=host64(s0), dfinal_state=dS.f64)
    ref = dict(zip(NAMES, (ref[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dinitial_state"))))

    def loss(out, S):
        return (host64(out) * dout.f64).sum() + (host64(S) * dS.f64).sum()

    out, S = od.delta_forward(**{n: host64(x) for n, x in base.items()})
    noise = 2 * 2.0 ** -18 * (np.linalg.norm(out) * np.linalg.norm(dout.f64) + np.linalg.norm(S) * np.linalg.norm(dS.f64))
    rows = np.abs((f64(f)["q"] * ref["q"]).sum(-1)) + np.abs((f64(f)["k"] * ref["k"]).sum(-1))
    for name in NAMES:
        x = base[name]
        size = torch.exp2(torch.floor(torch.log2(x.double().abs().clamp_min(2.0 ** -60))) - 7) if x.dtype == torch.bfloat16 \
            else x.double().abs() * 2.0 ** -8
        d = size * torch.from_numpy(np.sign(grads[name]))
        moved = [(x.double() + s * d).to(x.dtype) for s in (1, -1)]
        step = host64(moved[0]) - host64(moved[1])
        gpu, exact = [], []
        for m in moved:
            at = {**base, name: m}
            gpu.append(loss(*R.ret_delta_forward_chunkwise(**cuda(at), out_dtype=torch.float32, want_final_state=True)))
            o, s = od.delta_forward(**{n: host64(t) for n, t in at.items()})
            exact.append((o * dout.f64).sum() + (s * dS.f64).sum())
        third = exact[0] - exact[1] - (ref[name] * step).sum()
        change = (grads[name] * step).sum()
        own = np.linalg.norm(grads[name]) + (np.linalg.norm(rows) * (H // Hk) if name == "g" else 0)
        tol = noise + 2.0 ** -17 * own * np.linalg.norm(step)
        # the difference is above what it may be off by (a step of 2^-8 of a slow head's g hardly is)
        assert name == "g" or abs(change) > 2 * tol, (name, change, tol)
        assert abs(gpu[0] - gpu[1] - change - third) < tol, (name, gpu[0] - gpu[1], change, third, tol)
