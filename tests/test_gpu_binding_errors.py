"""Errors of the entry points that the direct binding calls: raised, with nothing
done twice."""
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
