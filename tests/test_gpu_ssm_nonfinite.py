"""Infinite and NaN operands of the selective scan and the causal convolution
on the GPU: what the formulas keep finite stays finite, and right, whatever
stands in other channels, groups, sequences and padding."""

import pytest

torch = pytest.importorskip("torch")
gcb = pytest.importorskip("grouped_convolution_backward_amd")

import ssm_reference as ref  # noqa: E402
from test_gpu_ssm import (_conv_case, _nan, _nan_bytes, _ref_conv, _ref_scan, _run_scan, _scan_case,  # noqa: E402
                          _seq_start)

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


def same(name, a, b):
    assert torch.equal(a, b), f"{name}: {int((a != b).sum())} of {a.numel()} values differ"


def _same_where_finite(got, want, scale, dtype, L, C, T):
    """Outputs are finite exactly where the 64-bit form is, and there within its bound."""
    terms = {"dB": C, "dC": C, "dA": T, "dD": T, "ddelta_bias": T}
    for k, v in got.items():
        kind = "fp32" if k in ("final_state", "dinit_state", "dA", "dD", "ddelta_bias") else dtype
        g, w, s = v.double().cpu().reshape(-1), want[k].reshape(-1), scale[k].reshape(-1)
        fine = torch.isfinite(w)
        assert torch.equal(torch.isfinite(g), fine), f"{k}: {int((torch.isfinite(g) != fine).sum())} of {g.numel()} values"
        ref.assert_close(k, g[fine], w[fine], s[fine], kind, 4 * L + 64 + terms.get(k, 128))


@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("dtype,C,S,G,segments", [("bf16", 40, 16, 2, 3), ("fp32", 262, 8, 2, 3), ("fp32", 36, 40, 3, 2),
                                                  ("bf16", 70, 16, 2, 0)])
def test_a_gradient_that_is_not_finite_stays_in_its_group(dtype, C, S, G, segments, value):
    """dy of channel 0 in the last segment: its group's dB and dC, its own gradients in rows before, and nothing else. Channels
    past the end of another group's last block must not carry it there."""
    c, p, starts, T = _scan_case(dtype, C, S, G, 1, 150, None, True, True)
    plan = gcb.ScanPlan(p, segments=segments, segments_backward=segments)
    print(f"[gpu] scan {p} {plan.info}", flush=True)
    clean = _run_scan(plan, c, starts, T)
    c["dy"][T - 2, 0] = value
    got = _run_scan(plan, c, starts, T)
    for k in ("dB", "dC"):
        same(k, got[k][:, 1:], clean[k][:, 1:])
        assert not bool(torch.isfinite(got[k][T - 2, 0]).any()), k
    for k in ("dx", "ddelta", "dz", "dinit_state"):
        same(k, got[k][:, 1:], clean[k][:, 1:])
    for k in ("dA", "dD", "ddelta_bias"):
        same(k, got[k][1:], clean[k][1:])
    for k in ("y", "final_state"):
        same(k, got[k], clean[k])
    want, scale = _ref_scan(c, starts)
    _same_where_finite(got, want, scale, dtype, 150, C, T)


@pytest.mark.parametrize("lens,segments", [(None, 0), (None, 2), ([90, 0, 61, 1, 35], 2)])
@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("name", ["x", "delta", "B", "C", "z", "dy", "init", "dfinal"])
def test_one_value_that_is_not_finite(name, value, lens, segments):
    """In one sequence, in one row or state: finite exactly where the 64-bit form is, forward and backward, in every output."""
    N = 5 if lens else 2
    c, p, starts, T = _scan_case("fp32", 70, 13, 2, N, 90, lens, True, True)
    if name in ("init", "dfinal"):
        c[name][N // 2, 3, 5] = value
    else:
        row = starts[N // 2] + 40
        c[name].view(T, -1)[row, 3] = value
    plan = gcb.ScanPlan(p, segments=segments, segments_backward=segments)
    print(f"[gpu] scan {name} = {value}, {p}", flush=True)
    got = _run_scan(plan, c, starts, T)
    want, scale = _ref_scan(c, starts)
    _same_where_finite(got, want, scale, "fp32", 90, 70, T)


@pytest.mark.parametrize("dtype,S,segments", [("fp32", 16, 0), ("fp32", 13, 2), ("bf16", 40, 2)])
def test_a_rate_of_minus_infinity_keeps_nothing(dtype, S, segments):
    """Such a state is d x B of the row alone: in the last row too, whose tile ends past the sequence, and in the gradients,
    where it counts as the lowest finite rate."""
    L = 75
    c, p, starts, T = _scan_case(dtype, 20, S, 1, 2, L, None, True, True)
    c["A"][3, 5], c["A"][7, 0] = -INF, -3e38
    plan = gcb.ScanPlan(p, segments=segments, segments_backward=segments)
    got = _run_scan(plan, c, starts, T)
    limit = dict(c, A=c["A"].clamp(min=-1e30))
    want, scale = _ref_scan(limit, starts)
    _same_where_finite(got, want, {k: v.nan_to_num() for k, v in scale.items()}, dtype, L, 20, T)
    state = torch.randn(2, 20, S, generator=torch.Generator().manual_seed(1)).cuda()
    y = torch.empty(2, 20, dtype=ref.TORCH[dtype], device="cuda")
    d = {k: v.cuda() for k, v in c.items()}
    plan.run_step(d["x"][:2], d["delta"][:2], d["A"], d["B"][:2], d["C"][:2], state, y, D=d["D"], z=d["z"][:2],
                  delta_bias=d["bias"])
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(state).all())


def _growing(S, L, segments):
    c, p, starts, T = _scan_case("fp32", 24, S, 1, 1, L, None, True, True)
    c["delta"].fill_(1.0)
    c["bias"].zero_()
    c["A"] = -c["A"].abs().clamp(max=4.0)
    c["A"][:, ::2] = 2.8                                    # over 32 rows e^89.6, above what fp32 holds
    plan = gcb.ScanPlan(dict(p, softplus=False), segments=segments, segments_backward=segments)
    assert plan.info["segments"] == plan.info["segments_backward"] and (plan.info["segments"] > 1) == (segments > 1)
    return c, starts, T, plan


@pytest.mark.parametrize("S,segments", [(16, 1), (16, 4), (5, 3), (40, 4), (100, 2)])
def test_growing_states_that_are_still_zero(S, segments):
    """Rates above 0 over segments whose decays multiply to more than fp32 holds, while the state (from its start) and its
    gradient (from its end) are still 0: a split must not make NaN of infinity times 0."""
    L = 120
    c, starts, T, plan = _growing(S, L, segments)
    c["x"][:100], c["dy"][20:] = 0.0, 0.0
    c["init"].zero_()
    c["dfinal"].zero_()
    got = _run_scan(plan, c, starts, T)
    want, scale = _ref_scan(c, starts, softplus=False)
    _same_where_finite(got, want, scale, "fp32", L, 24, T)


@pytest.mark.parametrize("S,segments", [(16, 1), (16, 2), (5, 2), (40, 2), (100, 2)])
def test_growing_states_from_very_small_ones(S, segments):
    """The same from a state of 1e-36, and a gradient of it: 60 rows end below 1e38, though one segment's decays alone
    multiply to more than fp32 holds."""
    L = 60
    c, starts, T, plan = _growing(S, L, segments)
    c["C"] *= 0.01
    c["init"].fill_(1e-36)
    c["x"].zero_()
    c["dy"].zero_()
    c["dfinal"].zero_()
    want, scale = _ref_scan(c, starts, softplus=False)
    got = _run_scan(plan, c, starts, T)
    assert float(want["final_state"].max()) > 1e36
    _same_where_finite(got, want, scale, "fp32", L, 24, T)
    c["init"].zero_()
    c["dfinal"].fill_(1e-36)
    c["B"] *= 0.01
    want, scale = _ref_scan(c, starts, softplus=False)
    got = _run_scan(plan, c, starts, T)
    assert float(want["dinit_state"].max()) > 1e36
    _same_where_finite(got, want, scale, "fp32", L, 24, T)


@pytest.mark.parametrize("lens", [None, [40, 0, 33, 1, 2, 38]])
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("name", ["x", "dy", "init", "dfinal", "w", "bias"])
@pytest.mark.parametrize("dtype,C,W,act", [("bf16", 36, 4, "silu"), ("fp32", 7, 8, "silu"), ("fp16", 1, 3, "none")])
def test_one_value_of_the_convolution_that_is_not_finite(dtype, C, W, act, name, value, lens):
    """Finite exactly where the 64-bit form is, in every output of forward and backward."""
    N, L = (6, 40) if lens else (3, 40)
    c, p, starts, T = _conv_case(dtype, C, W, N, L, lens, act, True, 0)
    at = {"x": (starts[2] + 12, C - 1), "dy": (starts[2] + 12, C - 1), "init": (2, W - 2, C - 1), "dfinal": (2, W - 2, C - 1),
          "w": (C - 1, 1), "bias": (C - 1,)}[name]
    c[name][at] = value
    want, scale = _ref_conv(c, starts, act)
    plan = gcb.CausalConvPlan(p)
    print(f"[gpu] conv {name} = {value}, {p}", flush=True)
    d = {k: v.cuda() for k, v in c.items()}
    seq = {"seq_start": _seq_start(starts)} if lens else {}
    y, final, dx = _nan(T, C, dtype=dtype), _nan(N, W - 1, C, dtype=dtype), _nan(T, C, dtype=dtype)
    dw, db, dinit = _nan(C, W), _nan(C), _nan(N, W - 1, C, dtype=dtype)
    plan.run(d["x"], d["w"], y, bias=d["bias"], init_state=d["init"], final_state=final, **seq)
    plan.run_backward(d["x"], d["w"], d["dy"], dx, dw, dbias=db, bias=d["bias"], init_state=d["init"], dinit_state=dinit,
                      dfinal_state=d["dfinal"], ws=_nan_bytes(plan.workspace_bytes), **seq)
    torch.cuda.synchronize()
    got = {"y": y, "final_state": final, "dx": dx, "dinit_state": dinit, "dw": dw, "dbias": db}
    for k, v in got.items():
        g, w, s = v.double().cpu().reshape(-1), want[k].reshape(-1), scale[k].reshape(-1)
        fine = torch.isfinite(w)
        assert torch.equal(torch.isfinite(g), fine), f"{k}: {int((torch.isfinite(g) != fine).sum())} of {g.numel()} values"
        if k == "final_state":
            same(k, g[fine], w[fine])
        else:
            ref.assert_close(k, g[fine], w[fine], s[fine], "fp32" if k in ("dw", "dbias") else dtype, 2 * W + 24 + T)
