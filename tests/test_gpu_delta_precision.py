"""What the chunked gated delta rule keeps of its numbers where a norm over
everything does not show it: bf16 outputs, states and gradients behind strong
decays.  The formats' bounds are those of the parity tests."""
import pytest
import torch

from tests.test_gpu_delta import cuda, inputs

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
