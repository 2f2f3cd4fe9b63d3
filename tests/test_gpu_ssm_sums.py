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
from test_gpu_ssm import _nan, _nan_bytes, _run_scan, _scan_case  # noqa: E402

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


@pytest.mark.parametrize("N,L,C,W", [(65536, 8, 64, 4), (4096, 64, 256, 4), (1, 2 ** 18, 4, 3)])
def test_convolution_parameter_gradients_over_many_rows(N, L, C, W):
    g = torch.Generator().manual_seed(N + L)
    x, dy = torch.randn(N, L, C, generator=g), torch.randn(N, L, C, generator=g)
    w, b = torch.randn(C, W, generator=g) * 0.6, torch.randn(C, generator=g) * 0.3
    plan = gcb.CausalConvPlan({"dtype": "fp32", "N": N, "L": L, "C": C, "W": W, "activation": "silu"})
    dx, dw, db = _nan(N, L, C), _nan(C, W), _nan(C)
    print(f"[gpu] conv {plan.problem}", flush=True)
    plan.run_backward(x.cuda(), w.cuda(), dy.cuda(), dx, dw, dbias=db, bias=b.cuda(), ws=_nan_bytes(plan.workspace_bytes))
    torch.cuda.synchronize()
    line = torch.cat([torch.zeros(N, W - 1, C), x], 1).double()
    p = b.double() + sum(line[:, k:k + L] * w[:, k].double() for k in range(W))
    s = dy.double() * ref.dsilu(p)
    want = torch.stack([(s * line[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)
    off = {"dw": _off(dw, want), "dbias": _off(db, s.sum((0, 1)))}
    print(off, flush=True)
    assert off["dw"] < 4e-7 and off["dbias"] < 4e-7, off
