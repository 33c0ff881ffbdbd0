"""The short calls' direct binding, host side: an error of the entry point is
raised, never tried again the general way (a decode step would be applied twice);
and the module's file belongs to the torch that it was built against."""
import importlib.util
import os

import pytest
import torch

import linear_recurrent_sequence_chunkwise_b200 as R

CALLS = {
    "delta_decode_step": lambda t: R.ret_delta_decode_step(t, t, t, t, t, t),
    "delta_forward": lambda t: R.ret_delta_forward_chunkwise(t, t, t, t, t),
    "delta_backward": lambda t: R.ret_delta_backward_chunkwise(t, t, t, t, t, t),
    "layernorm_forward": lambda t: R.ret_layernorm_forward(t),
    "layernorm_backward": lambda t: R.ret_layernorm_backward(t, t, t, t),
    "rotary": lambda t: R.ret_rotary(t, freqs=t),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_an_error_of_the_entry_point_is_raised_once(monkeypatch, name):
    calls = []
    monkeypatch.setattr(R._binding, name, lambda *a: calls.append(a) or R.RET_ERR_CUDA)
    monkeypatch.setattr(R, "_call", lambda *a: pytest.fail("called again the general way"))
    with pytest.raises(R.RetentionError) as e:
        CALLS[name](torch.zeros(2, 2))
    assert e.value.status == R.RET_ERR_CUDA and len(calls) == 1


@pytest.mark.parametrize("name", sorted(CALLS))
def test_what_the_binding_does_not_take_goes_the_general_way(monkeypatch, name):
    monkeypatch.setattr(R._binding, name, lambda *a: None)
    with pytest.raises((ValueError, TypeError)):  # a CPU tensor of two dimensions
        CALLS[name](torch.zeros(2, 2))


def test_the_file_is_the_running_torchs(monkeypatch):
    path = R._binding.__file__
    assert os.path.basename(path) == f"_binding-torch{torch.__version__}.so"
    spec = importlib.util.spec_from_file_location("_retention_build", os.path.join(os.path.dirname(path), "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    assert build.binding_path() == path
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert build.binding_path() != path and not os.path.exists(build.binding_path())


def test_a_missing_file_says_what_to_do(tmp_path):
    with pytest.raises(ImportError, match="build.py"):
        R._load_binding(str(tmp_path / "_binding-torch0.so"))
