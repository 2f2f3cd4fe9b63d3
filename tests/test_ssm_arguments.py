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


@pytest.mark.parametrize("shape,want,fits", [
    ((4, 3, 8), (4, 3, 8), True), ((12, 8), (4, 3, 8), True), ((1, 12, 1, 8), (4, 3, 8), True), ((96,), (4, 3, 8), True),
    ((2, 2, 3, 8), (4, 3, 8), True), ((4, 24), (4, 3, 8), True),
    ((3, 4, 8), (4, 3, 8), False),                       # rows of the sequences in turn
    ((4, 8, 3), (4, 3, 8), False), ((8, 12), (12, 8), False), ((24, 4), (12, 8), False),
    ((8, 1, 4), (8, 4), True), ((4, 8), (8, 4), False),  # [C, 1, W] and [W, C]
    ((6, 2, 16), (6, 2, 16), True), ((6, 32), (6, 2, 16), True), ((6, 16, 2), (6, 2, 16), False),
    ((6, 16), (6, 1, 16), True), ((1, 5), (5, 1), True), ((4, 3, 7), (4, 3, 8), False), ((0, 7), (0, 3, 8), True), ((1,), (1, 1, 1), True),
])
def test_shapes_that_hold_the_elements_in_order(shape, want, fits):
    from grouped_convolution_backward_amd import ssm
    assert ssm._same_order(shape, want) is fits
