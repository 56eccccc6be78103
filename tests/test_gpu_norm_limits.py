"""The head norm where its activation's argument is far from zero: a masked gate (the type's lowest value, minus
infinity) lets nothing through, the largest lets all through, in both directions."""

import math

import pytest
import torch

from oracle import seq_ref as R
from weight_linear_attention_gb300 import falcon as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = R.U
# Beyond 14 the bounds' relative errors (some units and 2 |v| of them, the argument's own rounding carried through
# the exponential) no longer grow: from 150 on e^-|v| is 0 in fp32 or its reciprocal is, so that every factor is
# exactly its limit (0 or 1, times v). Between 14 and 150 the gates below have no values.
FAR = 14.0
# The lower values give a factor of 0 and a slope of 0, the upper ones v (sigmoid: 1) and 1 (sigmoid: 0).
LOW = [None, -1e30, -1000.0, -150.0]  # None: the type's lowest, or largest
HIGH = [None, 1e30, 1000.0, 150.0]


def _values(values, dt, sign):
    return [sign * torch.finfo(dt).max if v is None else v for v in values]


def _close(name, got, ref, bound):
    ok, share = R.close(got, ref, bound)
    print(f"PARITY {name}: {share:.3f} of the bound")
    assert ok, f"{name}: {share:.3f} of the bound"


@pytest.fixture
def near(monkeypatch):
    """The reference's bounds with the arguments' size cut at FAR."""
    act, slope = R._act_error, R._slope_error
    monkeypatch.setattr(R, "_act_error", lambda name, v: act(name, v.clamp(-FAR, FAR)))
    monkeypatch.setattr(R, "_slope_error", lambda name, v: slope(name, v.clamp(-FAR, FAR)))


def _inputs(dt, seed, shape=(2, 2, 9, 64)):
    r = torch.Generator().manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    B, H, T, d = shape
    # small parameters and gradients: n times the type's largest value stays finite
    return (draw(*shape).to(dt), draw(*shape).to(dt), 0.05 * draw(H, d), 0.02 * draw(H, d), (0.05 * draw(*shape)).to(dt))


def _run(x, z, w, b, dy, act):
    dev = [None if t is None else t.cuda() for t in (x, z, w, b, dy)]
    y = F.groupnorm_forward(dev[0], dev[2], dev[3], dev[1], act=act)
    return y, F.groupnorm_backward(dev[0], dev[4], dev[2], dev[3], dev[1], act=act)


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_masked_gates(act, dt, near):
    """Whole rows and single channels of gates so low that nothing passes: exact zeros, the sums without them."""
    t = DT[dt]
    x, z, w, b, dy = _inputs(t, 1)
    low = torch.zeros(x.shape, dtype=torch.bool)
    for i, v in enumerate(_values(LOW, t, -1)):
        z[:, :, 1 + i] = v
        z[:, :, 6:, 11 + 9 * i] = v
        low[:, :, 1 + i] = low[:, :, 6:, 11 + 9 * i] = True
    y, got = _run(x, z, w, b, dy, act)
    assert not y.cpu()[low].any() and not got["dz"].cpu()[low].any()
    assert not got["dx"].cpu()[:, :, 1:5].any()
    _close("y", y, *R.gn_forward(x, w, b, z, act))
    ref, e = R.gn_backward(x, dy, w, b, z, act)
    for k in ref:
        _close(k, got[k], ref[k], e[k])


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_open_gates(act, dt, near):
    """The largest gates, one to a row and a channel so that no sum overflows."""
    t = DT[dt]
    x, z, w, b, dy = _inputs(t, 2)
    for i, v in enumerate(_values(HIGH, t, 1)):
        z[i // 2, i % 2, 5, 20 + i] = v
    y, got = _run(x, z, w, b, dy, act)
    _close("y", y, *R.gn_forward(x, w, b, z, act))
    ref, e = R.gn_backward(x, dy, w, b, z, act)
    for k in ref:
        _close(k, got[k], ref[k], e[k])


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_infinite_gates(act, dt, near):
    """What the formulas give: v s(v) is NaN at minus infinity (0 times it), the sigmoid 0 and 1."""
    t = DT[dt]
    x, z, w, b, dy = _inputs(t, 3)
    z[:, :, 2, 7], z[:, :, 4, 9], z[:, :, 4, 50] = -math.inf, math.inf, math.nan
    y, got = _run(x, z, w, b, dy, act)
    _close("y", y, *R.gn_forward(x, w, b, z, act))
    ref, e = R.gn_backward(x, dy, w, b, z, act)
    _close("dz", got["dz"], ref["dz"], e["dz"])
    rows = [0, 1, 3, 5, 6, 7, 8]
    _close("dx", got["dx"][:, :, rows], ref["dx"][:, :, rows], e["dx"][:, :, rows])


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("v", [-100.0, -95.0, -90.0, -88.0, -87.0, -60.0, -20.0])
def test_gates_around_the_smallest_exponential(act, v):
    """A logistic below 2^-126 may come out as zero, so v s(v) may be off by |v| 2^-126, and so may its slope; for the
    rest the reference's own bounds."""
    x, z, w, b, dy = _inputs(torch.float32, 4)
    z[:, :, 3] = v
    y, got = _run(x, z, w, b, dy, act)
    n = R._norm(x, w, b, 1e-5)[4]
    ref, e = R.gn_forward(x, w, b, z, act)
    _close("y", y, ref, e + abs(v) * 2.0 ** -126 * n.abs())
    ref, e = R.gn_backward(x, dy, w, b, z, act)
    _close("dz", got["dz"], ref["dz"], e["dz"] + abs(v) * 2.0 ** -126 * (n * dy.double()).abs())


@pytest.mark.parametrize("act", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_far_normalised_values(act, dt):
    """Without a gate the activation's argument is the normalised value: here the bias alone (weight 0)."""
    t = DT[dt]
    x, _, w, b, dy = _inputs(t, 5)
    low, high = _values(LOW, t, -1), _values(HIGH, t, 1)
    for i, v in enumerate(low + high):
        w[:, 3 + 5 * i], b[:, 3 + 5 * i] = 0.0, v
    y, got = _run(x, None, w, b, dy, act)
    total = dy.double().sum((0, 2))
    # every addend of dbias is dy times 0 or 1 (a unit or two off); at most 18 rows and 40 additions in a row
    room = (18 + 40 + 4) * U * dy.double().abs().sum((0, 2))
    for i, v in enumerate(low + high):
        c = 3 + 5 * i
        f = 0.0 if v < 0 else 1.0 if act == "sigmoid" else v
        df = 1.0 if v > 0 and act != "sigmoid" else 0.0
        want = torch.full(y.shape[:3], f, dtype=torch.double)
        _close(f"y {v}", y[..., c], want, 4 * U * want)
        _close(f"dbias {v}", got["dbias"][:, c], df * total[:, c], df * room[:, c])
    assert got["dx"].isfinite().all() and got["dweight"].isfinite().all()
