"""Calls of the causal convolution and the selective scan as programs make
them: the single calls on the current stream and on another one, while the
current one goes on allocating; against the plans' own results."""

import pytest

torch = pytest.importorskip("torch")
gcb = pytest.importorskip("grouped_convolution_backward_amd")

import ssm_reference as ref  # noqa: E402
from test_gpu_ssm import _check_scan, _conv_case, _ref_conv, _ref_scan, _scan_case  # noqa: E402

pytestmark = pytest.mark.gpu


def _busy(stream):
    """A few milliseconds of work on a stream, so that what is enqueued behind it starts later than the host goes on."""
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-4
    return a


@pytest.mark.parametrize("how", ["current", "stream", "handle"])
def test_single_calls_with_their_own_workspace(how):
    """A split scan, whose segment sums are in a workspace that the call itself allocates, and a convolution: on another
    stream, memory that the current stream gets meanwhile must not be theirs."""
    C, L = 64, 2000
    c, p, starts, T = _scan_case("bf16", C, 16, 1, 1, L, None, True, True)
    assert gcb.ScanPlan(p).workspace_bytes > 0
    cc, cp, cstarts, _ = _conv_case("bf16", C, 4, 1, L, None, "silu", True, 0)
    d = {k: v.cuda() for k, v in c.items()}
    dc = {k: v.cuda() for k, v in cc.items()}
    side = torch.cuda.Stream()
    stream = {"current": None, "stream": side, "handle": side.cuda_stream}[how]
    torch.cuda.synchronize()
    keep = _busy(side) if stream is not None else None
    kw = {} if stream is None else {"stream": stream}
    y = gcb.selective_scan(p, d["x"], d["delta"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"], delta_bias=d["bias"],
                           init_state=d["init"], **kw)
    u = gcb.causal_conv(cp, dc["x"], dc["w"], bias=dc["bias"], init_state=dc["init"], **kw)
    # the current stream fills whatever the allocator has free for it
    for n in (gcb.ScanPlan(p).workspace_bytes, y.numel() * 2, u.numel() * 2):
        for _ in range(8):
            torch.full((n // 4,), float("nan"), device="cuda")
    if stream is not None:
        torch.cuda.current_stream().wait_stream(side)
    y, u = y.clone(), u.clone()
    torch.cuda.synchronize()
    del keep
    want, scale = _ref_scan(c, starts, grads=False)
    _check_scan({"y": y}, want, scale, "bf16", L, C, T)
    want, scale = _ref_conv(cc, cstarts, "silu", grads=False)
    ref.assert_close("y", u, want["y"], scale["y"], "bf16", 32)
