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


def _refused(call, *names):
    """Every operand in `names`, with its last two axes exchanged (as many elements, another order), is a ValueError that
    names it; the call itself is none."""
    base = call.keywords
    call()
    for name in names:
        bad = base[name].transpose(-1, -2).contiguous()
        assert bad.shape != base[name].shape, name
        with pytest.raises(ValueError, match=f"^{name}: "):
            call(**{name: bad})
    torch.cuda.synchronize()


def test_operands_of_another_shape_are_refused():
    from functools import partial
    N, L, C, W, G, S = 2, 10, 12, 4, 3, 5

    def t(*shape):
        return torch.zeros(*shape, device="cuda")

    conv = gcb.CausalConvPlan({"dtype": "fp32", "N": N, "L": L, "C": C, "W": W})
    rows = {k: t(N, L, C) for k in ("x", "y")}
    states = {k: t(N, W - 1, C) for k in ("init_state", "final_state")}
    _refused(partial(conv.run, w=t(C, W), **rows, **states), "x", "y", "w", "init_state", "final_state")
    rows = {k: t(N, L, C) for k in ("x", "dy", "dx")}
    states = {k: t(N, W - 1, C) for k in ("init_state", "dinit_state", "dfinal_state")}
    _refused(partial(conv.run_backward, w=t(C, W), dw=t(C, W), ws=conv.new_workspace(), **rows, **states),
             "x", "dy", "dx", "w", "dw", "init_state", "dinit_state", "dfinal_state")
    _refused(partial(conv.run_step, x=t(2, C), w=t(C, W), state=t(7, W - 1, C), y=t(2, C)), "x", "w", "state", "y")

    scan = gcb.ScanPlan({"dtype": "fp32", "N": N, "L": L, "C": C, "G": G, "S": S})
    ins = {**{k: t(N, L, C) for k in ("x", "delta", "z")}, **{k: t(N, L, G, S) for k in ("B", "C")}, "A": t(C, S)}
    saved, ws = scan.new_saved(), scan.new_workspace()
    _refused(partial(scan.run, y=t(N, L, C), init_state=t(N, C, S), final_state=t(N, C, S), saved=saved, ws=ws, **ins),
             "x", "delta", "z", "B", "C", "A", "y", "init_state", "final_state")
    outs = {**{k: t(N, L, C) for k in ("dy", "dx", "ddelta", "dz")}, **{k: t(N, L, G, S) for k in ("dB", "dC")}, "dA": t(C, S)}
    _refused(partial(scan.run_backward, saved=saved, ws=ws, dinit_state=t(N, C, S), dfinal_state=t(N, C, S), **ins, **outs),
             "x", "delta", "z", "B", "C", "A", "dy", "dx", "ddelta", "dz", "dB", "dC", "dA", "dinit_state", "dfinal_state")
    one = {**{k: t(4, C) for k in ("x", "delta", "z", "y")}, **{k: t(4, G, S) for k in ("B", "C")}, "A": t(C, S)}
    _refused(partial(scan.run_step, state=t(6, C, S), **one), "x", "delta", "z", "y", "B", "C", "A", "state")


def test_operands_of_merged_and_split_axes():
    """The same elements in the same order: rows of all sequences in one axis, one more axis of 1, G and S merged."""
    N, L, C, W, G, S = 2, 10, 12, 4, 3, 5
    g = torch.Generator().manual_seed(3)

    def t(*shape):
        return torch.randn(*shape, generator=g).cuda()

    conv = gcb.CausalConvPlan({"dtype": "fp32", "N": N, "L": L, "C": C, "W": W})
    x, w = t(N, L, C), t(C, W)
    want, got = torch.zeros_like(x), torch.zeros_like(x)
    conv.run(x, w, want)
    conv.run(x.view(N * L, C), w.view(C, 1, W), got.view(1, N * L, C))
    assert torch.equal(got, want) and bool(want.any())
    scan = gcb.ScanPlan({"dtype": "fp32", "N": N, "L": L, "C": C, "G": G, "S": S})
    A, b, c = -t(C, S).abs(), t(N, L, G, S), t(N, L, G, S)
    scan.run(x, x, A, b, c, want, ws=scan.new_workspace())
    scan.run(x.view(-1, C), x, A, b.view(N * L, G * S), c.view(N * L, G, S), got, ws=scan.new_workspace())
    torch.cuda.synchronize()
    assert torch.equal(got, want) and bool(want.any())


@pytest.mark.parametrize("dtype,C", [("bf16", 40), ("fp16", 33), ("fp32", 6), ("bf16", 5)])
def test_operands_that_lie_on_an_element_only(dtype, C):
    """Every operand of the convolution, its states too, one element past a vector's alignment."""
    N, L, W = 3, 37, 4
    c, p, starts, T = _conv_case(dtype, C, W, N, L, None, "silu", True, 0)
    want, scale = _ref_conv(c, starts, "silu")

    def off(t, kind=dtype):
        whole = torch.full((t.numel() + 9,), float("nan"), dtype=ref.TORCH[kind], device="cuda")
        inner = whole[1:1 + t.numel()].view(t.shape)
        inner.copy_(t.cuda())
        return whole, inner

    ins = {k: off(v)[1] for k, v in c.items()}
    outs = {k: off(torch.full(s, float("nan"))) for k, s in
            {"y": (T, C), "final_state": (N, W - 1, C), "dx": (T, C), "dinit_state": (N, W - 1, C)}.items()}
    sums = {k: off(torch.full(s, float("nan")), "fp32") for k, s in {"dw": (C, W), "dbias": (C,)}.items()}
    plan = gcb.CausalConvPlan(p)
    print(f"[gpu] conv {p}", flush=True)
    plan.run(ins["x"], ins["w"], outs["y"][1], bias=ins["bias"], init_state=ins["init"], final_state=outs["final_state"][1])
    plan.run_backward(ins["x"], ins["w"], ins["dy"], outs["dx"][1], sums["dw"][1], dbias=sums["dbias"][1], bias=ins["bias"],
                      init_state=ins["init"], dinit_state=outs["dinit_state"][1], dfinal_state=ins["dfinal"], ws=plan.new_workspace())
    torch.cuda.synchronize()
    for k, (whole, inner) in {**outs, **sums}.items():
        assert bool(torch.isnan(whole[:1]).all()) and bool(torch.isnan(whole[1 + inner.numel():]).all()), k
        if k == "final_state":
            assert torch.equal(inner.double().cpu(), want[k])
        else:
            ref.assert_close(k, inner, want[k], scale[k], "fp32" if k in sums else dtype, 2 * W + 24 + (T if k in sums else 0))
