"""Outputs that the calls make themselves on a stream that the caller passes."""
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


def calls():
    x, dy = torch.randn(600, 512, device="cuda").bfloat16(), torch.randn(600, 512, device="cuda").bfloat16()
    _, mean, rstd = R.ret_layernorm_forward(x, want_stats=True)
    yield "layernorm_forward", lambda s: R.ret_layernorm_forward(x, want_stats=True, stream=s)
    yield "layernorm_backward", lambda s: R.ret_layernorm_backward(dy, x, mean, rstd, stream=s)
    q, k = torch.randn(2, 70, 4, 64, device="cuda"), torch.randn(2, 70, 2, 64, device="cuda")
    yield "rotary", lambda s: R.ret_rotary(q, k, freqs=R.ret_rotary_frequencies(64)[0], stream=s)
    f, s0 = inputs(981, 2, 130, 2, 4, 64, 72, "bf16")
    c, s0 = cuda(f), s0.cuda()
    yield "delta_forward", lambda s: R.ret_delta_forward_chunkwise(**c, initial_state=s0, want_final_state=True, stream=s)
    yield "delta_backward", lambda s: R.ret_delta_backward_chunkwise(**c, dout=c["v"], initial_state=s0, stream=s)
    one = {n: t[:, 0].contiguous() for n, t in c.items()}
    states = [s0.clone(), s0.clone()]  # there before the stream that is kept waiting
    yield "delta_decode_step", lambda s: R.ret_delta_decode_step(**one, state=states.pop(), stream=s)


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_are_not_in_use_on_another_stream(handle):
    """Memory of every size that the call needs is freed on the current stream while
    work there is still to write it; the call's outputs, on another stream, are not
    that memory."""
    s = torch.cuda.Stream()
    for name, call in calls():
        want = call(None)
        want = list(want) if isinstance(want, tuple) else [want]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        busy = [torch.empty_like(t) for t in want for _ in range(4) if t is not None]
        for t in busy:
            t.fill_(7)
        del busy, t
        got = call(s.cuda_stream if handle else s)
        got = list(got) if isinstance(got, tuple) else [got]
        torch.cuda.synchronize()
        for a, b in zip(want, got, strict=True):
            assert a is b is None or torch.equal(a, b), name
