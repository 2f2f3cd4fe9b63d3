"""Launches of more than 2^24 workgroups of 256, that is 2^32 work items, which
one axis of a grid cannot hold: as many short sequences, rows of single tokens,
and rows of B and C to join. Inputs with few rows that are not 0, or all the
same, so that the results are exact."""

import pytest

torch = pytest.importorskip("torch")
gcb = pytest.importorskip("grouped_convolution_backward_amd")

pytestmark = pytest.mark.gpu

MANY = 2 ** 24 + 3
F32 = torch.float32


def _few(n, seed):
    """n values, 0 but for the first and the last eight rows."""
    t = torch.zeros(n, 1, device="cuda")
    v = torch.randint(1, 9, (16,), generator=torch.Generator().manual_seed(seed)).float().cuda()
    t[:8, 0], t[-8:, 0] = v[:8], v[8:]
    return t


def _nan(*shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def test_convolution_of_many_sequences():
    x, dy, w = _few(MANY, 1), _few(MANY, 2), torch.tensor([[2.0, 3.0, 5.0]], device="cuda")
    plan = gcb.CausalConvPlan({"dtype": "fp32", "N": MANY, "L": 1, "C": 1, "W": 3, "activation": "none"})
    y, final = _nan(MANY, 1), _nan(MANY, 2, 1)
    print("[gpu] conv forward", flush=True)
    plan.run(x, w, y, final_state=final)
    torch.cuda.synchronize()
    assert torch.equal(y, 5 * x) and torch.equal(final[:, 1], x) and not bool(final[:, 0].any())
    dx, dw, db = _nan(MANY, 1), _nan(1, 3), _nan(1)
    print("[gpu] conv backward", flush=True)
    plan.run_backward(x, w, dy, dx, dw, dbias=db, ws=plan.new_workspace())
    torch.cuda.synchronize()
    assert torch.equal(dx, 5 * dy)
    assert dw.tolist() == [[0.0, 0.0, float((x * dy).double().sum())]] and float(db) == float(dy.double().sum())


def test_scan_of_many_sequences_and_rows():
    x, dy, one = _few(MANY, 3), _few(MANY, 4), torch.ones(MANY, 1, device="cuda")
    A = torch.zeros(1, 1, device="cuda")
    plan = gcb.ScanPlan({"dtype": "fp32", "N": MANY, "L": 1, "C": 1, "S": 1, "softplus": False})
    y, saved, ws = _nan(MANY, 1), plan.new_saved(), plan.new_workspace()
    print("[gpu] scan forward", flush=True)
    plan.run(x, one, A, one, one, y, saved=saved, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, x)
    out = {k: _nan(MANY, 1) for k in ("dx", "ddelta", "dB", "dC")}
    dA, dD, dbias = _nan(1, 1), _nan(1), _nan(1)
    print("[gpu] scan backward", flush=True)
    plan.run_backward(x, one, A, one, one, dy, saved, dA=dA, dD=dD, ddelta_bias=dbias, ws=ws, **out)
    torch.cuda.synchronize()
    assert torch.equal(out["dx"], dy)
    for k in ("ddelta", "dB", "dC"):
        assert torch.equal(out[k], x * dy), k
    assert float(dA) == 0 and float(dD) == float(dbias) == float((x * dy).double().sum())
    state = one.clone().view(MANY, 1, 1)
    print("[gpu] scan step", flush=True)
    plan.run_step(x, one, A, one, one, state, y)
    torch.cuda.synchronize()
    assert torch.equal(y, x + 1) and torch.equal(state.view(MANY, 1), y)


def test_scan_with_many_values_of_b_and_c():
    """2^16 groups of 128 states: 256 rows have 2^32 sums of dB and dC."""
    T, G, S = 256, 2 ** 16, 128
    one = torch.ones(T, G, dtype=torch.bfloat16, device="cuda")
    bc = torch.ones(T, G, S, dtype=torch.bfloat16, device="cuda")
    A = torch.zeros(G, S, device="cuda")
    plan = gcb.ScanPlan({"dtype": "bf16", "N": 1, "L": T, "C": G, "G": G, "S": S, "softplus": False})
    y, saved, ws = torch.empty_like(one), plan.new_saved(), plan.new_workspace()
    print("[gpu] scan of 2^16 groups", flush=True)
    plan.run(one, one, A, bc, bc, y, saved=saved, ws=ws)
    dx, dd, dA = torch.empty_like(one), torch.empty_like(one), _nan(G, S)
    dB, dC = torch.zeros_like(bc), torch.zeros_like(bc)
    plan.run_backward(one, one, A, bc, bc, one, saved, dx, dd, dA, dB, dC, ws=ws)
    torch.cuda.synchronize()
    row = torch.arange(T, device="cuda").to(torch.bfloat16).view(T, 1, 1)
    assert bool((dC == row + 1).all()) and bool((dB == T - row).all())
    assert bool((y == (row + 1).view(T, 1) * S).all())
