"""The gated delta rule's calls beside each other on several streams, in every
form of the chain: blocks of four, two and one groups of columns, bf16 and fp32
outputs, and the gradients.  Calls that share the GPU wait longer for each other
within a block (tiles come late, warps poll, a warp's last reads of a stage come
late); the results are the same bits as a call's alone."""
import pytest
import torch

from retention_inputs import make_tensor
from tests.helpers import dev
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


def beside_each_other(calls, rounds):
    """Each of four streams runs all calls, from another one on, ``rounds`` times."""
    want = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(rounds):
        got = []
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got.append([calls[(i + j) % len(calls)]() for j in range(len(calls))])
        torch.cuda.synchronize()
        for i, results in enumerate(got):
            for j, result in enumerate(results):
                for n, (a, b) in enumerate(zip(result, want[(i + j) % len(calls)], strict=True)):
                    assert torch.equal(a, b), ((i + j) % len(calls), n)


# B, N, Hk, H, dk, dv.  Sixteen heads of four sequences fill the SMs with blocks of
# four groups of columns (two with an fp32 output); one or two sequences of few
# heads get blocks of two and one.
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shapes", [
    [(4, 330, 8, 16, 128, 128), (4, 200, 16, 16, 256, 72), (4, 400, 8, 16, 64, 136), (5, 130, 16, 16, 128, 72)],
    [(2, 400, 4, 8, 128, 200), (1, 500, 4, 4, 256, 96), (3, 300, 2, 6, 64, 200), (1, 300, 1, 2, 256, 40)],
])
def test_prompts(shapes, out_dtype):
    calls = []
    for B, N, Hk, H, dk, dv in shapes:
        f, s0 = inputs(931, B, N, Hk, H, dk, dv, "bf16")
        c, s0 = cuda(f), s0.cuda()
        calls.append(lambda c=c, s0=s0: R.ret_delta_forward_chunkwise(**c, initial_state=s0, out_dtype=out_dtype,
                                                                      want_final_state=True))
    beside_each_other(calls, 60)


# Blocks of two groups of columns, the last shape's of one.  The second shape's
# blocks leave room on an SM for those of other calls, which hold a warp up most.
def test_gradients():
    calls = []
    for B, N, Hk, H, dk, dv in ((4, 200, 8, 16, 128, 128), (3, 300, 2, 6, 64, 200), (4, 130, 8, 16, 256, 40),
                                 (1, 700, 2, 4, 128, 96)):
        f, s0 = inputs(932, B, N, Hk, H, dk, dv, "bf16")
        c, s0, dout = cuda(f), s0.cuda(), dev(make_tensor(932, 4, (B, N, H, dv), "bf16"))
        calls.append(lambda c=c, s0=s0, dout=dout: R.ret_delta_backward_chunkwise(**c, dout=dout, initial_state=s0,
                                                                                 dfinal_state=s0))
    beside_each_other(calls, 200)
