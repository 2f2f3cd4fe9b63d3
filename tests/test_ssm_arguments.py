"""Arguments of the causal convolution and the selective scan that do not fit,
without a GPU."""

import pytest

import grouped_convolution_backward_amd as gcb


@pytest.mark.parametrize("N,L,T", [(1, 0, 5), (3, 4, 13), (2, 2 ** 20, 2 ** 21 + 1)])
def test_packed_rows_that_no_sequence_can_hold_are_refused(N, L, T):
    """Rows past every sequence of at most L rows would stay unwritten."""
    base = {"dtype": "bf16", "N": N, "L": L, "T": T, "C": 8, "packed": True}
    for make, kw in ((gcb.CausalConvPlan, {"W": 4}), (gcb.ScanPlan, {"S": 4})):
        with pytest.raises(gcb.WgradError, match="T must be at most N") as e:
            make({**base, **kw}, hip_device=-1)
        assert e.value.code == gcb.ERR_INVALID_ARG
        make({**base, **kw, "T": N * L}, hip_device=-1)
