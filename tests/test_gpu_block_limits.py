"""Where the gated delta rule and the root-mean-square norm can go wrong beside their parity: what a call's parts leave for one
another, values that are not finite, operands' bits, decays of every strength."""

import math

import pytest
import torch

from oracle import block_ref as R
from tests.test_gpu_block import DT, backward, forward, inputs
from weight_linear_attention_gb300 import falcon as F

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(8, 12, 1024, 64, 64), (4, 8, 1024, 128, 128), (6, 9, 500, 64, 128)], ids=str)
def test_gdr_maps_leave_in_order(dt, size):
    """A chunk's tiles leave shared memory one after another, in planes and then as fp32, while the next is formed in their
    place: calls in a row, beside copies that keep the memory busy, have the same bits."""
    p, _ = inputs(*size, DT[dt], 1)
    busy = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())  # its memory may have been a call's until now
    out, S = forward(p)
    for _ in range(20):
        with torch.cuda.stream(side):
            busy[1 << 27:].copy_(busy[:1 << 27])
        o, s = forward(p)
        assert torch.equal(o, out) and torch.equal(s, S)
    torch.cuda.synchronize()


def near(what, got, want, dtype=torch.float32, room=R.NEAR, size=None):
    share = R.gdr_near(got, want, dtype, room, size)
    print(f"NEAR {what}: {share:.3f} of the bound")
    assert share <= 1, f"{what}: {share:.3f} of the bound"


LONG = [(2, 2, 33, 64, 64), (2, 2, 200, 64, 64), (1, 2, 130, 40, 100), (1, 3, 500, 128, 128), (1, 1, 2500, 64, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", LONG, ids=str)
def test_gdr_forward_keeps_fp32s_bits(dt, size):
    """Operands of 16 bits in the place of 24 would not pass: test_block_host.py shows it of the bound."""
    p, _ = inputs(*size, DT[dt], 40)
    out, S = forward(p)
    ro, rs = R.gdr_forward(**p)
    near("out", out, ro, DT[dt])
    near("S_final", S, rs)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", LONG, ids=str)
@pytest.mark.parametrize("shared", [False, True])
def test_gdr_backward_keeps_fp32s_bits(dt, size, shared):
    p, a = inputs(*size, DT[dt], 41, 1 if shared else None)
    got = backward(p, a)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    for name in ("dq", "dk", "dv", "dbeta", "dS0"):
        near(name, got[name], want[name], DT[dt] if name in ("dq", "dk", "dv") else torch.float32)
    near("dg", got["dg"], want["dg"], room=R.NEAR_DG, size=terms_of_dg(p, a, want))


@pytest.mark.parametrize("size", [(1, 2, 156, 128, 128), (2, 1, 459, 32, 128), (2, 3, 66, 100, 64), (1, 2, 300, 64, 64)], ids=str)
def test_gdr_sums_of_products_keep_fp32s_bits(size):
    """Results that are sums of products (two blocks of a wide head, dk's four terms): half of the bound, 16 U, which is one and
    a half of the 11 U that it stands on. Small products that were added to a whole sum left 12 to 20 U."""
    p, a = inputs(*size, torch.float32, 46)
    out, S = forward(p)
    got = dict(backward(p, a), out=out, S_final=S)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    want["out"], want["S_final"] = R.gdr_forward(**p)
    for name in ("out", "S_final", "dq", "dk", "dv", "dbeta", "dS0"):
        near(name, got[name], want[name], room=R.NEAR / 2)


def terms_of_dg(p, a, want):
    """The norm of what dg is summed from: dq.q (of heads that share a key each for itself) and dv.v."""
    q, k = (p[x].repeat_interleave(p["v"].shape[1] // p[x].shape[1], 1) for x in ("q", "k"))
    own = R.gdr_backward(q, k, p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])["dq"]
    return torch.stack([(own * q).sum(-1), (want["dv"] * p["v"]).sum(-1)]).square().sum((0, -1)).sqrt()


BAD = [("v", math.nan), ("v", math.inf), ("k", math.nan), ("k", -math.inf), ("q", math.nan), ("q", math.inf),
       ("beta", math.nan), ("beta", math.inf), ("g", math.nan), ("g", math.inf)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,dk,dv", [(20, 64, 64), (130, 64, 64), (200, 128, 72)])
@pytest.mark.parametrize("name,value", BAD, ids=lambda x: str(x))
def test_gdr_tokens_before_a_value_that_is_not_finite(dt, T, dk, dv, name, value):
    """Each head has one such value at another token: what the definition makes of it is not finite either, all else is, and
    right."""
    at = [t for t in (0, 3, 15, 16, 17, 31, 33, 47, 48, 63, 64, 79, 100, T - 1) if t < T]
    p, _ = inputs(1, len(at), T, dk, dv, DT[dt], 42)
    for h, t in enumerate(at):
        if p[name].dim() == 4:
            p[name][0, h, t, 5] = value
        else:
            p[name][0, h, t] = value
    out, S = forward(p)
    ro, rs = R.gdr_forward(**p)
    for got, want, dtype in ((out.cpu(), ro, DT[dt]), (S.cpu(), rs, torch.float32)):
        there = torch.isfinite(want)
        assert torch.equal(torch.isfinite(got), there)
        ok, share = R.gdr_close(torch.where(there, got, 0), torch.where(there, want, 0), R.GDR, dtype)
        assert ok, share


STRONG = [-3.9, -4.5, -6.0, -9.0, -12.0, -20.0, -60.0, -80.0]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,dk,dv", [(20, 64, 64), (150, 64, 64), (100, 128, 40), (130, 48, 100), (90, 128, 128)])
def test_gdr_dg_of_strong_decays(dt, T, dk, dv):
    """All tokens of a head decay alike, down to e^-80: the error of dg is one of dg itself."""
    p, a = inputs(2, len(STRONG), T, dk, dv, DT[dt], 43)
    p["g"] = torch.tensor(STRONG)[None, :, None].expand(2, -1, T).contiguous()
    got = backward(p, a)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    for h, g in enumerate(STRONG):
        # above -4 a difference of terms that are e^3.9 as great
        room = R.NEAR_DG * (math.exp(3.9) if g > -4 else 1)
        near(f"dg at {g}", got["dg"][:, h:h + 1], want["dg"][:, h:h + 1], room=room)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", [-1.9, -2.1])
def test_gdr_dg_on_both_sides_of_its_rule(dt, d, g):
    p, a = inputs(1, 4, 200, d, d, DT[dt], 45)
    p["g"] = torch.full_like(p["g"], g)
    got = backward(p, a)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    near("dg", got["dg"], want["dg"], room=R.NEAR_DG, size=terms_of_dg(p, a, want) if g > -2 else None)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [False, True])
def test_gdr_dg_of_strong_decays_among_weak_ones(dt, shared):
    """Every seventh token forgets (and one in a sequence that ends early, gains of 0 beside it): its dg by itself."""
    T, n = 300, torch.tensor([300, 170], dtype=torch.int32)
    p, a = inputs(2, len(STRONG), T, 64, 64, DT[dt], 44, 2 if shared else None)
    strong = torch.arange(T) % 7 == 3
    p["g"] = torch.where(strong, torch.tensor(STRONG)[:, None], torch.tensor(-0.05)).expand(2, -1, -1).contiguous()
    p["beta"][:, :, 5::14] = 0
    p["g"][0, :, 101] = -math.inf
    got = backward(p, a, n)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"], lengths=n)
    assert not got["dg"][0, :, 101].any() and not got["dg"][1, :, 170:].any()
    for h, g in enumerate(STRONG):
        room = R.NEAR_DG * (math.exp(3.9) if g > -4 else 1)
        near(f"dg at {g}", got["dg"][:, h:h + 1, strong], want["dg"][:, h:h + 1, strong], room=room)
        weak = ~strong & (torch.arange(T) != 101)
        near(f"dg beside {g}", got["dg"][:, h:h + 1, weak], want["dg"][:, h:h + 1, weak], room=R.NEAR_DG)


@pytest.mark.parametrize("d", [100, 768, 4096, 8200])
def test_rms_8_bits_are_those_of_the_quotient(d):
    """Value by value: the fp32 call's y by the scale, rounded once more. Rows of every size, one with an infinity."""
    r = torch.Generator().manual_seed(d)
    x = torch.randn(1, 4000, d, generator=r).cuda()
    x[0, 7] = 0
    w = torch.randn(d, generator=r) * 2.0 ** torch.randint(-20, 20, (d,), generator=r)
    for w in (w, w * 1e31, w * 1e-32, w * 1e-36):
        y, _, _ = F.rmsnorm_forward(x, w.cuda())
        y8, _, s = F.rmsnorm_forward(x, w.cuda(), out_dtype=torch.float8_e4m3fn)
        top = y.abs().amax(-1)
        # the scale is the nearest fp32 value of the largest |y| / 448 but for subnormal ones (torch multiplies by 1 / 448 where
        # 448 is a number)
        assert torch.equal(s, top / torch.full_like(top, 448)) if top[top > 0].min() > 1e-35 else torch.allclose(s, top / 448, rtol=1e-6, atol=1e-44)
        want = torch.where(s[..., None] > 0, y / s[..., None], 0.0).clamp(-448, 448).to(torch.float8_e4m3fn)
        assert torch.equal(y8.view(torch.uint8) & 0x7f, want.view(torch.uint8) & 0x7f) and torch.equal(y8.float(), want.float())
    w = torch.ones(d)
    w[3] = math.inf
    y8, _, s = F.rmsnorm_forward(x[:, :5], w.cuda(), out_dtype=torch.float8_e4m3fn)
    y8 = y8.float()
    assert torch.isinf(s).all() and torch.isnan(y8[..., 3]).all() and not y8[..., :3].any() and not y8[..., 4:].any()
