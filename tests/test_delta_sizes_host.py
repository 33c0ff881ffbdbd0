"""Sizes that the gated delta rule's entry points refuse because an index would not
hold them."""
import pytest

import linear_recurrent_sequence_chunkwise_b200 as R
from tests.test_abi_host import needs_no_gpu
from tests.test_delta_host import INVALID, backward, refused


@needs_no_gpu
@pytest.mark.parametrize("Hk,dv,fits", [(1, 520, False), (3, 1544, False), (1, 504, True), (5, 2504, True)])
def test_value_columns_of_a_key_head(Hk, dv, fits):
    """A chunk's rows of all value heads of a key head are counted in 32 bits."""
    H = 65535
    refused(backward(B=1, N=64, Hk=Hk, H=H, dv=dv, nbytes=1), INVALID)  # the workspace is too small in any case
    assert (H // Hk * dv < 1 << 25) == fits
    assert ("2^25" in R.ret_last_error_string()) == (not fits)
