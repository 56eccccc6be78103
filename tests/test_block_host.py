"""Host-only checks of the gated delta rule and the root-mean-square norm: their references against differences, and
calls that the synchronous argument check refuses, or that have nothing to do, so that nothing is launched."""

import math

import pytest
import torch

from oracle import block_ref as R
from weight_linear_attention_gb300 import build as fbuild
from weight_linear_attention_gb300 import falcon as F

A = 1 << 40  # fake device addresses: never dereferenced
GB = 1 << 30
OK, INV, UNS, MIS = F.FALCON_OK, F.FALCON_ERR_INVALID_ARG, F.FALCON_ERR_UNSUPPORTED, F.FALCON_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def lib():
    fbuild.build()
    return F.load()


# ---- the references


def _gdr_inputs(B=2, H=4, Hk=2, T=5, dk=3, dv=4):
    r = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.double)  # noqa: E731
    k = n(B, Hk, T, dk)
    return dict(q=n(B, Hk, T, dk), k=k / k.norm(dim=-1, keepdim=True), v=n(B, H, T, dv),
                beta=torch.sigmoid(n(B, H, T)), g=-torch.exp(n(B, H, T) - 1), S0=n(B, H, dk, dv)), n


@pytest.mark.parametrize("lengths", [None, torch.tensor([5, 2], dtype=torch.int32)])
def test_delta_rule_gradients_by_differences(lengths):
    p, n = _gdr_inputs()
    dout, dS = n(2, 4, 5, 4), n(2, 4, 3, 4)

    def loss(p):
        out, S = R.gdr_forward(**p, lengths=lengths)
        return (out * dout).sum() + (S * dS).sum()

    got = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], dout, p["S0"], dS, lengths=lengths)
    for name in p:
        step, d = n(*p[name].shape), 1e-6
        up, down = (loss(dict(p, **{name: p[name] + s * step})) for s in (d, -d))
        want = (up - down) / (2 * d)
        assert abs((got["d" + name] * step).sum() - want) < 1e-7 * (1 + abs(want)), name


def test_delta_rule_by_hand():
    # one head, dk = dv = 1: S = a S + k beta (v - a S k)
    one = lambda x: torch.tensor(x, dtype=torch.double).view(1, 1, -1, 1)  # noqa: E731
    out, S = R.gdr_forward(one([2., 1.]), one([1., 0.5]), one([3., 4.]), one([0.5, 1.])[..., 0],
                           one([math.log(0.5), 0.])[..., 0], torch.full((1, 1, 1, 1), 2.0), scale=1.0)
    # token 0: kept 1, error 3 - 1, S = 1 + 0.5 * 2 = 2, out 4; token 1: kept 2, error 4 - 1, S = 2 + 0.5 * 3 = 3.5
    assert out.flatten().tolist() == pytest.approx([4.0, 3.5]) and S.item() == pytest.approx(3.5)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_bound_sees_operands_of_16_bits(dt):
    """The bound of a whole head in its norm: a state, or any input, cut to 16 bits goes past it in what is made of it."""
    r = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=r)  # noqa: E731
    B, H, T, d = 2, 2, 70, 64
    p = dict(q=n(B, H, T, d), k=n(B, H, T, d), v=n(B, H, T, d).to(dt), beta=torch.sigmoid(n(B, H, T)),
             g=-torch.exp(n(B, H, T) - 3), S0=n(B, H, d, d) / 8)
    p["q"], p["k"] = ((x / x.norm(dim=-1, keepdim=True)).to(dt) for x in (p["q"], p["k"]))
    out, S = R.gdr_forward(**p)
    assert R.gdr_near(out.to(dt), out, dt) < 1 and R.gdr_near(S.float(), S) < 1
    for name in ("S0", "beta") if dt == torch.bfloat16 else ("q", "k", "v", "S0", "beta"):
        o, s = R.gdr_forward(**dict(p, **{name: R.cut(p[name], 16)}))
        t = 20 if name == "S0" else T  # little is left of it behind
        assert R.gdr_near(o[:, :, :t].to(dt), out[:, :, :t], dt) > 1, name
        if name in ("k", "v", "beta"):
            assert R.gdr_near(s.float(), S) > 1, name


def test_norm_gradients_by_differences():
    r = torch.Generator().manual_seed(2)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.double)  # noqa: E731
    h, w, dy, dh = n(2, 3, 7), n(7), n(2, 3, 7), n(2, 3, 7)
    (dx, dw), _ = R.rms_backward(h, dy, w, dh, eps=0.1)
    loss = lambda h, w: (R.rms_forward(h, w, eps=0.1)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    d = 1e-6
    s = n(2, 3, 7)
    assert abs((dx * s).sum() - (loss(h + d * s, w) - loss(h - d * s, w)) / (2 * d)) < 1e-7
    s = n(7)
    assert abs((dw * s).sum() - (loss(h, w + d * s) - loss(h, w - d * s)) / (2 * d)) < 1e-7


def test_e4m3_values():
    x = torch.randn(4000, generator=torch.Generator().manual_seed(3)) * torch.logspace(-4, 2, 4000)
    x = x.clamp(-448, 448)
    assert torch.equal(R.e4m3(x.double()), x.to(torch.float8_e4m3fn).double())


# ---- refusals of the delta rule


def _dims(b=2, h=4, hk=2, t=40, dk=64, dv=32, dtype=F.FALCON_BF16):
    return F.make_gdr_dims(b, h, t, dk, dv, qk_heads=hk, dtype=dtype)


def fwd(dims=None, strides=None, scale=1.0, ws=A + 20 * GB, ws_bytes=None, **kw):
    dims = dims or _dims()
    p = dict(q=A, k=A + GB, v=A + 2 * GB, beta=A + 3 * GB, g=A + 4 * GB, S0=None, lengths=None, out=A + 5 * GB,
             S_final=None)
    p.update(kw)
    n = F.falcon_gdr_workspace_bytes(dims) if ws_bytes is None else ws_bytes
    return F.falcon_gdr_fwd(*p.values(), dims, strides, scale, ws, n, stream=0)


def bwd(dims=None, strides=None, scale=1.0, ws=A + 20 * GB, ws_bytes=None, **kw):
    dims = dims or _dims()
    p = dict(q=A, k=A + GB, v=A + 2 * GB, beta=A + 3 * GB, g=A + 4 * GB, S0=None, lengths=None, dout=A + 5 * GB,
             dS_final=None, dq=A + 6 * GB, dk=A + 7 * GB, dv=A + 8 * GB, dbeta=A + 9 * GB, dg=A + 10 * GB, dS0=None)
    p.update(kw)
    n = F.falcon_gdr_workspace_bytes(dims, True) if ws_bytes is None else ws_bytes
    return F.falcon_gdr_bwd(*p.values(), dims, strides, scale, ws, n, stream=0)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("dims,want", [
    (_dims(b=-1), INV), (_dims(h=-2), INV), (_dims(hk=-1), INV), (_dims(t=-1), INV), (_dims(dk=0), INV),
    (_dims(dv=0), INV), (_dims(hk=3), INV), (_dims(hk=0), INV), (_dims(hk=8), INV), (_dims(dtype=2), UNS),
    (_dims(dk=129), UNS), (_dims(dv=129), UNS), (_dims(t=1 << 30), UNS), (_dims(b=1 << 31), UNS),
    (_dims(b=1 << 27, h=2, hk=2), UNS), (_dims(b=1 << 12, h=1 << 8, hk=1 << 8, t=1 << 17), UNS),
])
def test_delta_rule_sizes(call, dims, want):
    assert call(dims=dims) == want
    assert F.falcon_gdr_workspace_bytes(dims) == 0 and F.falcon_gdr_workspace_bytes(dims, True) == 0


def test_delta_rule_nothing_to_do():
    for d in (_dims(b=0), _dims(h=0, hk=0), _dims(h=0)):
        assert fwd(dims=d, ws=None) == OK and bwd(dims=d, ws=None) == OK
    d = _dims()
    d.reserved = 1
    assert fwd(dims=d) == INV
    assert F.load().falcon_gdr_workspace_bytes(None, 0) == 0
    for s in (math.nan, math.inf, -math.inf):
        assert fwd(scale=s) == INV and bwd(scale=s) == INV


def test_delta_rule_takes_every_finite_scale():
    for x in (3.4028234e38, -3.4028234e38, 1e-45, 0.0):
        assert fwd(dims=_dims(b=0), ws=None, scale=x) == OK and bwd(dims=_dims(b=0), ws=None, scale=x) == OK


def test_delta_rule_missing_and_misaligned():
    for name in ("q", "k", "v", "beta", "g", "out"):
        assert fwd(**{name: None}) == INV, name
    for name in ("q", "k", "v", "beta", "g", "dout", "dq", "dk", "dv", "dbeta", "dg"):
        assert bwd(**{name: None}) == INV, name
    for name in ("q", "k", "v", "out"):
        assert fwd(**{name: A + 11 * GB + 1}) == MIS, name
    for name in ("beta", "g", "S0", "lengths", "S_final"):
        assert fwd(**{name: A + 11 * GB + 2}) == MIS, name
    for name in ("dbeta", "dg", "dS_final", "dS0"):
        assert bwd(**{name: A + 11 * GB + 2}) == MIS, name


def test_delta_rule_workspace():
    n, m = F.falcon_gdr_workspace_bytes(_dims()), F.falcon_gdr_workspace_bytes(_dims(), True)
    assert 0 < n < m and n % 256 == 0 and m % 256 == 0
    assert fwd(ws=None) == INV and bwd(ws=None) == INV
    assert fwd(ws_bytes=n - 1) == INV and bwd(ws_bytes=m - 1) == INV
    assert fwd(ws=A + 20 * GB + 128) == MIS
    assert fwd(ws=A + 5 * GB) == INV and bwd(ws=A + 2 * GB) == INV  # on a tensor
    for t in (0, 1, 32):
        assert F.falcon_gdr_workspace_bytes(_dims(t=t)) == 0
    assert F.falcon_gdr_workspace_bytes(_dims(t=33)) > 0
    # shared heads need their partial gradients
    assert F.falcon_gdr_workspace_bytes(_dims(hk=4), True) < m


def test_delta_rule_segments():
    """Whether a sequence is cut shows in the workspace: two scans side by side fill the GPU with half the sequences."""
    kib, up = 1024, lambda n: (n + 255) // 256 * 256  # noqa: E731

    def uncut(bh, chunks, tiles, rows, bwd):  # X, M, A, S; dA, dS
        per = 24 + 24 * tiles * tiles + 16 * tiles * rows + (16 + 24) * tiles * rows * bwd
        return up(bh * chunks * per * kib) + up(bh * (chunks + 1) * 24 * tiles * rows * kib)

    def whole(bh, chunks, d, bwd):
        n = F.falcon_gdr_workspace_bytes(_dims(b=1, h=bh, hk=bh, t=64 * chunks, dk=d, dv=d), bwd)
        least = uncut(bh, chunks, (d + 63) // 64, (d + 63) // 64, bwd)
        assert n >= least
        return n == least

    # 64 chunks of one scan, a step 1.5 us alone on an SM and 2.6 where two share it: 96 us uncut
    assert whole(48, 64, 64, True) and whole(16, 128, 128, True)
    assert whole(96, 16, 64, False) and whole(96, 16, 64, True)
    assert not whole(2, 64, 64, True) and not whole(12, 1024, 64, False) and not whole(12, 1024, 64, True)


def test_delta_rule_written_buffers_overlap_nothing():
    assert fwd(out=A) == INV and fwd(S_final=A + 5 * GB) == INV
    assert fwd(S0=A + 11 * GB, S_final=A + 11 * GB + 16) == INV
    assert bwd(dq=A + 7 * GB) == INV and bwd(dbeta=A + 3 * GB) == INV
    assert bwd(S0=A + 11 * GB, dS0=A + 11 * GB) == INV
    dense = [2 * 40 * 64, 40 * 64, 64] * 2 + [4 * 40 * 32, 40 * 32, 32] + [160, 40, 1] * 2
    assert fwd(strides=dense + [0, 40 * 32, 32]) == INV
    assert fwd(strides=dense + [4 * 40 * 32, 40 * 32, -32]) == INV
    assert fwd(strides=dense[:9] + [160, 40, -1] + dense[12:] + [4 * 40 * 32, 40 * 32, 32]) == INV


# ---- refusals of the norm


def _rms(b=2, t=5, d=64, dtype=F.FALCON_BF16, out=None):
    return F.make_rms_dims(b, t, d, dtype=dtype, out_dtype=out)


def norm(dims=None, strides=None, eps=1e-6, **kw):
    p = dict(x=A, residual=A + GB, weight=None, lengths=None, h=A + 2 * GB, y=A + 3 * GB, scales=None)
    p.update(kw)
    return F.falcon_rms_fwd(*p.values(), dims or _rms(), strides, eps, stream=0)


def norm_b(dims=None, strides=None, eps=1e-6, ws=A + 9 * GB, ws_bytes=1 << 30, **kw):
    p = dict(h=A, weight=None, lengths=None, dy=A + GB, dh=A + 2 * GB, dx=A + 3 * GB, dweight=A + 4 * GB)
    p.update(kw)
    return F.falcon_rms_bwd(*p.values(), dims or _rms(), strides, eps, ws, ws_bytes, stream=0)


@pytest.mark.parametrize("call", [norm, norm_b])
@pytest.mark.parametrize("dims,want", [
    (_rms(b=-1), INV), (_rms(t=-1), INV), (_rms(d=0), INV), (_rms(dtype=2), UNS), (_rms(out=F.FALCON_F32), UNS),
    (_rms(out=3), UNS), (_rms(d=16385), UNS), (_rms(b=1 << 16, t=1 << 15), UNS), (_rms(t=1 << 30), UNS),
])
def test_norm_sizes(call, dims, want):
    assert call(dims=dims) == want


def test_norm_arguments():
    for eps in (0.0, -1e-5, math.nan, math.inf):
        assert norm(eps=eps) == INV and norm_b(eps=eps) == INV
    for name in ("x", "y"):
        assert norm(**{name: None}) == INV, name
    for name in ("h", "dy", "dx"):
        assert norm_b(**{name: None}) == INV, name
    assert norm(residual=None) == INV                      # h without a sum to write
    assert norm(scales=A + 5 * GB) == INV                  # scales without 8 bits
    assert norm(dims=_rms(out=F.FALCON_E4M3)) == INV       # and 8 bits without scales
    assert norm_b(dims=_rms(out=F.FALCON_E4M3)) == UNS
    assert norm(x=A + 1) == MIS and norm(weight=A + 5 * GB + 2) == MIS
    assert norm_b(ws=None) == INV and norm_b(ws_bytes=F.falcon_rms_bwd_workspace_bytes(_rms()) - 1) == INV
    assert norm_b(ws=A + 9 * GB + 128) == MIS and norm_b(ws=A + 3 * GB) == INV


def test_norm_overlap():
    assert norm(y=A) == INV and norm(y=A + 2 * GB) == INV and norm(h=A + 16) == INV
    dense = [5 * 64, 64]
    assert norm(h=A, strides=dense + dense + [5 * 128, 128] + dense) == INV    # in place only where it is the same view
    assert norm(h=A + GB, strides=dense + [5 * 128, 128] + dense + dense) == INV
    assert norm_b(dx=A) == INV and norm_b(dx=A + GB) == INV
    assert norm_b(dx=A + 2 * GB, strides=dense + dense + [5 * 128, 128] + dense) == INV
    assert norm(strides=dense * 3 + [320, 32]) == INV and norm(strides=[-320, 64] + dense * 3) == INV


def test_norm_nothing_to_do():
    for d in (_rms(b=0), _rms(t=0)):
        assert norm(dims=d) == OK and F.falcon_rms_bwd_workspace_bytes(d) == 0
        assert norm_b(dims=d, dweight=None, ws=None) == OK


def test_wrappers_refuse_host_tensors():
    x = torch.zeros(1, 2, 20, 8)
    g = torch.zeros(1, 2, 20)
    for call in (lambda: F.gdr_forward(x, x, x, g, g), lambda: F.gdr_backward(x, x, x, g, g, x),
                 lambda: F.rmsnorm_forward(x[0]), lambda: F.rmsnorm_backward(x[0], x[0])):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match=r"\[B,T,d\]"):
        F.rmsnorm_forward(x)
    with pytest.raises(ValueError, match=r"\[B,H,T,d\]"):
        F.gdr_forward(x[0], x[0], x[0], g, g)
