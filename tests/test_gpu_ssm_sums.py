"""Accuracy of the parameters' gradients, which are sums over every row, for
long sequences and for many of them, in fp32 against 64 bits.

A running sum of n terms of either sign is off by about 0.42 x 2^-24 sqrt(n / 2)
of its size (roundings of half a unit at most, independent of each other): 16384
rows that 16 lanes sum one after another would give 5.7e-7. The kernels sum in
levels of some tens, three levels of which give 1e-7 to 2e-7; the terms' own
roundings, as large as the ones of dx and ddelta (1e-7 and 2.5e-7), add up to as
much relative to the sum, in squares. The bounds are twice what that comes to.
"""

import pytest

torch = pytest.importorskip("torch")
gcb = pytest.importorskip("grouped_convolution_backward_amd")

import ssm_reference as ref  # noqa: E402
from test_gpu_ssm import _conv_case, _nan, _nan_bytes, _run_scan, _scan_case  # noqa: E402

pytestmark = pytest.mark.gpu


def _off(got, want):
    got = got.double().cpu().reshape(want.shape)
    return float((got - want).norm() / want.norm())


@pytest.mark.parametrize("S,N,L", [(16, 1, 16384), (8, 1, 16384), (40, 1, 4096), (16, 700, 16)])
def test_scan_parameter_gradients_over_many_rows(S, N, L):
    c, p, starts, T = _scan_case("fp32", 64, S, 1, N, L, None, True, True)
    plan = gcb.ScanPlan(p, segments=1, segments_backward=1)
    print(f"[gpu] scan {p}", flush=True)
    got = _run_scan(plan, c, starts, T)
    d = {k: v.double() for k, v in c.items()}
    want = ref.scan(d["x"], d["delta"], d["A"], d["B"], d["C"], starts, d["D"], d["z"], d["bias"], d["init"], True, dy=d["dy"],
                    dfinal=d["dfinal"])
    off = {k: _off(got[k], want[k]) for k in ("dD", "ddelta_bias", "dA")}
    print(off, flush=True)
    assert off["dD"] < 4e-7 and off["ddelta_bias"] < 6e-7 and off["dA"] < 1e-6, off
