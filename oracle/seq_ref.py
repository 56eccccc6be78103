"""64-bit references of the strided [B,H,T,d] operators, token by token, with bounds on what fp32 arithmetic
may be off by.

Inputs are CPU tensors of any type; everything is computed in double from their values. Each function returns its
results and, for each, an elementwise bound of the rounding error of an evaluation in fp32 (unit roundoff
U = 2^-24) before the result is rounded to its own type. The bounds follow the computation: a quantity of relative
error r and magnitude m contributes r m, and errors are carried through the recurrences as the values are."""

import math

import torch

U = 2.0 ** -24


def half_step(dtype):
    """Largest relative error of rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def valid(lengths, B, T):
    """[B,1,T,1] truth values: the token lies inside its sequence."""
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    return (torch.arange(T)[None, :] < n[:, None])[:, None, :, None]


def gate(name, g):
    """a, 1 - a and the relative error that fp32 makes of either. The argument of the exponential carries its own
    rounding, |g| U relative to the result, the hardware's exponential and reciprocal two units each, the sums and
    products around them one each: 10 units and 2 |g|."""
    g = g.double()
    if name == "decay":
        a = torch.exp(g)
        om = -torch.expm1(g)
    else:
        a = torch.sigmoid(g)
        om = torch.sigmoid(-g)
    mag = torch.where(torch.isfinite(g), g.abs(), 0.0).clamp(max=200)
    return a, om, (10 + 2 * mag) * U


def glr_forward(name, x, g, h0=None, lengths=None):
    """(out, h_final), (bound of out, bound of h_final)."""
    B, H, T, d = x.shape
    a, om, ea = gate(name, g)
    ok = valid(lengths, B, T)
    x = torch.where(ok, x.double(), 0.0)
    a, om, ea = torch.where(ok, a, 1.0), torch.where(ok, om, 0.0), torch.where(ok, ea, 0.0)
    u = om * x if name == "mix" else x
    eu = (ea + U) * u.abs() if name == "mix" else torch.zeros_like(u)
    h = torch.zeros(B, H, d, dtype=torch.double) if h0 is None else h0.double()
    s, e = h.abs(), torch.zeros_like(h)  # magnitude of what is summed, bound of the error
    out, bound = torch.zeros(B, H, T, d, dtype=torch.double), torch.zeros(B, H, T, d, dtype=torch.double)
    for t in range(T):
        # a token adds the gate's error, the roundings of its own step (2) and, at most, those of composing maps
        # (3 more: the token's factor takes part in one product and one sum of a level, of at most three levels)
        grow = a[:, :, t] * s
        e = a[:, :, t] * e + (ea[:, :, t] + 5 * U) * grow + eu[:, :, t] + 2 * U * u[:, :, t].abs()
        s = grow + u[:, :, t].abs()
        h = a[:, :, t] * h + u[:, :, t]
        out[:, :, t], bound[:, :, t] = h, e
    return (torch.where(ok, out, 0.0), h), (torch.where(ok, bound, 0.0), e)


def glr_backward(name, x, g, out, dout, h0=None, dh_final=None, lengths=None):
    """(dx, dg, dh0) given the stored outputs `out`, and their bounds."""
    B, H, T, d = x.shape
    a, om, ea = gate(name, g)
    ok = valid(lengths, B, T)
    a, om, ea = torch.where(ok, a, 1.0), torch.where(ok, om, 0.0), torch.where(ok, ea, 0.0)
    x, dout, h = (torch.where(ok, v.double(), 0.0) for v in (x, dout, out))
    first = torch.zeros(B, H, 1, d, dtype=torch.double) if h0 is None else h0.double()[:, :, None]
    before = torch.cat([first, h[:, :, :-1]], 2)
    slope = before if name != "mix" else before - x
    f = (a if name == "decay" else a * om) * slope
    ef = (2 * ea + 4 * U) * f.abs()
    c = torch.zeros(B, H, d, dtype=torch.double) if dh_final is None else dh_final.double()
    s, e = c.abs(), torch.zeros_like(c)
    r = {k: torch.zeros(B, H, T, d, dtype=torch.double) for k in ("dx", "dg", "ex", "eg")}
    for t in reversed(range(T)):
        dh, mag = dout[:, :, t] + c, dout[:, :, t].abs() + s
        eh = e + 2 * U * mag
        if name == "mix":
            r["dx"][:, :, t] = om[:, :, t] * dh
            r["ex"][:, :, t] = om[:, :, t] * eh + (ea[:, :, t] + 2 * U) * om[:, :, t] * mag
        else:
            r["dx"][:, :, t], r["ex"][:, :, t] = dh, eh
        r["dg"][:, :, t] = dh * f[:, :, t]
        r["eg"][:, :, t] = eh * f[:, :, t].abs() + mag * (ef[:, :, t] + U * f[:, :, t].abs())
        c, s = a[:, :, t] * dh, a[:, :, t] * mag
        # where a is kept as 1 - (1 - a) its rounding is U, not a U: mag U
        e = a[:, :, t] * eh + (ea[:, :, t] + 5 * U) * s + (U * mag if name == "mix" else 0.0)
    keep = lambda v: torch.where(ok, v, 0.0)  # noqa: E731
    return (keep(r["dx"]), keep(r["dg"]), c), (keep(r["ex"]), keep(r["eg"]), e)


def act(name, v):
    """f(v), f'(v)."""
    if name == "none":
        return v, torch.ones_like(v)
    if name == "sigmoid":
        s = torch.sigmoid(v)
        return s, s * torch.sigmoid(-v)
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s + v * s * torch.sigmoid(-v)
    phi = 0.5 * torch.erfc(-v / math.sqrt(2))
    return v * phi, phi + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)


def _act_error(name, v):
    """Relative error of the activation's factor in fp32: as for a gate; Phi's argument v / sqrt 2 is rounded, which
    its tail magnifies by v^2."""
    if name == "none":
        return torch.zeros_like(v)
    if name == "gelu":
        return (12 + 2 * v * v) * U
    return (12 + 2 * v.abs()) * U


def _slope_error(name, v):
    """Absolute error of act'(v), its terms being of magnitude at most 1 + |v|."""
    return (0.0 if name == "none" else 16 * U) * (1 + v.abs()) + torch.zeros_like(v)


def _norm(x, weight, bias, eps):
    x = x.double()
    d = x.shape[-1]
    mu = x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (x - mu) * rstd
    # the mean: a row's sum is at most 32 + 5 additions deep, and 1 / d is rounded: 40 U of the largest |x|, which
    # moves xh by that much over the deviation; the variance's relative error is as large and the root halves it
    big = x.abs().amax(-1, keepdim=True)
    e = 42 * U * big * rstd + (32 * U) * xh.abs() + U * xh.abs()
    w = 1.0 if weight is None else weight.double()[None, :, None]
    b = 0.0 if bias is None else bias.double()[None, :, None]
    n = w * xh + b
    en = (abs(w) if weight is None else w.abs()) * (e + U * xh.abs()) + U * n.abs()
    return xh, e, rstd, w, n, en, d


def gn_forward(x, weight=None, bias=None, z=None, name="none", eps=1e-5, lengths=None):
    """y and its bound."""
    ok = valid(lengths, x.shape[0], x.shape[2])
    x = torch.where(ok, x.double(), 0.0)
    _, _, _, _, n, en, _ = _norm(x, weight, bias, eps)
    if z is None:
        y, df = act(name, n)
        e = (df.abs() + _slope_error(name, n)) * en + (_act_error(name, n) + 2 * U) * y.abs()
        # f'' is below 1.1 for every activation
        e = e + 0.6 * en ** 2
    else:
        z = torch.where(ok, z.double(), 0.0)
        f, _ = act(name, z)
        y = n * f
        e = en * f.abs() + (_act_error(name, z) + 2 * U) * y.abs()
    return torch.where(ok, y, 0.0), torch.where(ok, e, 0.0)


def gn_backward(x, dy, weight=None, bias=None, z=None, name="none", eps=1e-5, lengths=None):
    """dict dx, dz, dweight, dbias and a dict of their bounds."""
    B, H, T, d = x.shape
    ok = valid(lengths, B, T)
    x, dy = torch.where(ok, x.double(), 0.0), torch.where(ok, dy.double(), 0.0)
    xh, e, rstd, w, n, en, _ = _norm(x, weight, bias, eps)
    r, b = {}, {}
    if z is None:
        _, df = act(name, n)
        dn = dy * df
        edn = dy.abs() * (1.1 * en + _slope_error(name, n)) + U * dn.abs()
    else:
        z = torch.where(ok, z.double(), 0.0)
        f, df = act(name, z)
        dn = dy * f
        edn = (_act_error(name, z) + 2 * U) * dn.abs()
        r["dz"] = torch.where(ok, dy * n * df, 0.0)
        b["dz"] = torch.where(ok, dy.abs() * (en * df.abs() + n.abs() * _slope_error(name, z)) + 3 * U * r["dz"].abs(), 0.0)
    p = dn * w
    aw = abs(w) if weight is None else w.abs()
    ep = aw * edn + U * p.abs()
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    m1, m2 = mean(p), mean(p * xh)
    # sums at most 37 additions deep, 1 / d rounded
    e1 = mean(ep) + 40 * U * mean(p.abs())
    e2 = mean(ep * xh.abs() + p.abs() * e) + 41 * U * mean((p * xh).abs())
    dx = rstd * (p - m1 - xh * m2)
    size = p.abs() + m1.abs() + (xh * m2).abs()
    ex = rstd * (ep + e1 + xh.abs() * e2 + e * m2.abs() + 3 * U * size) + 36 * U * rstd * size
    r["dx"], b["dx"] = torch.where(ok, dx, 0.0), torch.where(ok, ex, 0.0)
    # every row's addend, and at most B T + 40 additions in a row
    add, eadd = dn * xh, edn * xh.abs() + dn.abs() * e
    deep = (B * T + 40) * U
    tot = lambda v: torch.where(ok, v, 0.0).sum((0, 2))  # noqa: E731
    r["dweight"], b["dweight"] = tot(add), tot(eadd) + deep * tot(add.abs())
    r["dbias"], b["dbias"] = tot(dn), tot(edn) + deep * tot(dn.abs())
    return r, b


def close(got, ref, bound):
    """(whether |got - ref| stays within the bound and the rounding to got's own type, everywhere; the largest share
    of it that was used). A result rounded to half a step of a value that is itself off by the bound. Where the
    reference is not finite, got has to be the same."""
    g = got.detach().cpu()
    half = half_step(g.dtype) if g.dtype != torch.float32 else U
    g = g.double()
    tiny = 2.0 ** -126  # below it the hardware's exponential gives zero
    room = bound * (1 + half) + half * ref.abs() + tiny
    fine = torch.isfinite(ref)
    same = torch.where(fine, True, (g == ref) | (g.isnan() & ref.isnan()))
    if not bool(same.all()):
        return False, math.inf
    share = torch.where(fine, (g - ref).abs() / room, 0.0)
    share = torch.nan_to_num(share, nan=math.inf)
    m = float(share.max()) if share.numel() else 0.0
    return m <= 1.0, m
