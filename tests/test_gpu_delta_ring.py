"""The gated delta rule's decode step on states of more than 64 MB, which a ring of
tiles of 32 columns takes through shared memory: every number of rows a thread has,
key widths below a thread's rows, a dv that ends inside a tile, shared key heads,
both types.  fp32 arithmetic: the suite's 1e-5; a bf16 output adds its rounding."""
import numpy as np
import pytest
import torch

from tests.helpers import host64
from tests.test_gpu_delta import TOL_F32

pytestmark = pytest.mark.gpu

R = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global R
    import linear_recurrent_sequence_chunkwise_b200 as mod
    R = mod
    yield mod
    mod.ret_check_device_error()


@pytest.mark.parametrize("B,Hk,H,dk,dv,dtype,out_dtype", [
    (96, 8, 16, 64, 200, torch.bfloat16, torch.float32),
    (250, 4, 16, 20, 256, torch.float32, torch.bfloat16),
    (80, 16, 16, 100, 164, torch.bfloat16, torch.bfloat16),
    (120, 8, 16, 128, 72, torch.float32, torch.float32),
    (41, 8, 16, 130, 200, torch.bfloat16, torch.float32),
    (30, 16, 32, 256, 76, torch.bfloat16, torch.bfloat16),
    (1000, 1, 1, 256, 68, torch.float32, torch.float32),
    (2100, 2, 4, 96, 20, torch.bfloat16, torch.float32),
])
def test_large_states(B, Hk, H, dk, dv, dtype, out_dtype):
    assert B * H * dk * dv * 4 >= 64e6
    gen = torch.Generator(device="cuda")
    gen.manual_seed(961)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    S = 0.3 * normal(B, H, dk, dv)
    ref = S.double()
    rep = H // Hk
    for _ in range(3):
        q, k = (normal(B, Hk, dk) / dk).to(dtype), torch.nn.functional.normalize(normal(B, Hk, dk), dim=-1).to(dtype)
        v, g, beta = normal(B, H, dv).to(dtype), -normal(B, H).abs(), normal(B, H).sigmoid()
        o = R.ret_delta_decode_step(q, k, v, g, beta, S, out_dtype=out_dtype)
        # the definition in 64 bits
        kd, qd = (x.double().repeat_interleave(rep, 1) for x in (k, q))
        ref *= g.double().exp()[..., None, None]
        u = beta.double()[..., None] * (v.double() - (kd[:, :, None] @ ref)[:, :, 0])
        ref += kd[..., None] * u[:, :, None]
        want = host64((qd[:, :, None] @ ref)[:, :, 0])
        got = host64(o)
        slack = TOL_F32 * np.linalg.norm(want, axis=-1, keepdims=True)
        if out_dtype == torch.float32:
            assert np.all(np.linalg.norm(got - want, axis=-1, keepdims=True) <= slack)
        else:
            assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + slack)
    err = (S - ref).flatten(2).norm(dim=-1) / ref.flatten(2).norm(dim=-1)
    assert float(err.max()) < TOL_F32
