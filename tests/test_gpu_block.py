"""GPU parity of the gated delta rule and the root-mean-square norm against their 64-bit references, within the rounding
bounds that oracle/block_ref.py derives."""

import math
import threading

import pytest
import torch

from oracle import block_ref as R
from oracle import seq_ref as SR
from weight_linear_attention_gb300 import falcon as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape):
        return torch.randn(*shape, generator=self.g)


def gpu(t):
    return None if t is None else t.cuda()


def inputs(B, H, T, dk, dv, dt, seed=1, Hk=None, S0=True):
    r = Draw(seed)
    Hk = H if Hk is None else Hk
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    p = dict(q=unit(r(B, Hk, T, dk)).to(dt), k=unit(r(B, Hk, T, dk)).to(dt), v=r(B, H, T, dv).to(dt),
             beta=torch.sigmoid(r(B, H, T)), g=-torch.exp(r(B, H, T) - 3))
    p["S0"] = r(B, H, dk, dv) / dk ** 0.5 if S0 else None
    return p, dict(dout=r(B, H, T, dv).to(dt), dS_final=r(B, H, dk, dv) / dk ** 0.5)


def place(layout, *tensors):
    """CPU tensors [B,Hi,T,(di)] on the GPU: dense, as column blocks of one [B,T,...] buffer ("blocks"), or one element
    off every vector boundary ("odd")."""
    if layout == "dense":
        return [t.cuda() for t in tensors]
    if layout == "odd":
        return [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) for t in tensors]
    rows = [t if t.dim() == 4 else t[..., None] for t in tensors]
    B, _, T, _ = rows[0].shape
    buf = torch.full((B, T, sum(t.shape[1] * t.shape[3] for t in rows)), math.nan, dtype=tensors[0].dtype, device="cuda")
    out, at = [], 0
    for t, src in zip(rows, tensors):
        n = t.shape[1] * t.shape[3]
        v = buf[:, :, at:at + n].unflatten(2, (t.shape[1], t.shape[3])).transpose(1, 2)
        v.copy_(t)
        out.append(v if src.dim() == 4 else v[..., 0])
        at += n
    return out


def forward(p, lengths=None, layout="dense", **kw):
    q, k, v = place(layout, p["q"], p["k"], p["v"])
    beta, g = place(layout, p["beta"], p["g"])
    if "out" not in kw:
        kw["out"], = place(layout, torch.full(p["v"].shape, math.nan, dtype=p["v"].dtype))
    return F.gdr_forward(q, k, v, beta, g, gpu(p["S0"]), lengths=gpu(lengths), **kw)


def backward(p, a, lengths=None, layout="dense", **kw):
    q, k, v, dout = place(layout, p["q"], p["k"], p["v"], a["dout"])
    beta, g = place(layout, p["beta"], p["g"])
    nan = lambda *names: place(layout, *(torch.full(p[n].shape, math.nan, dtype=p[n].dtype) for n in names))  # noqa: E731
    for names in (("q", "k", "v"), ("beta", "g")):
        for n, t in zip(names, nan(*names)):
            kw.setdefault("d" + n, t)
    return F.gdr_backward(q, k, v, beta, g, dout, gpu(p["S0"]), gpu(a["dS_final"]), lengths=gpu(lengths), **kw)


def check(what, got, want, room, dtype=torch.float32):
    ok, share = R.gdr_close(got, want, room, dtype)
    print(f"PARITY {what}: {share:.3f} of the bound")
    assert ok, f"{what}: {share:.3f} of the bound"


def check_forward(out, S, p, lengths=None, scale=None):
    dt = p["q"].dtype
    ro, rs = R.gdr_forward(**p, lengths=lengths, scale=scale)
    check("out", out, ro, R.GDR if dt == torch.float32 else R.GDR_BF16, dt)
    check("S_final", S, rs.flatten(2), R.GDR) if S.dim() == 3 else check("S_final", S.flatten(2), rs.flatten(2), R.GDR)


def check_backward(got, p, a, lengths=None, scale=None):
    dt = p["q"].dtype
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"],
                          lengths=lengths, scale=scale)
    for name in ("dq", "dk", "dv", "dbeta", "dg", "dS0"):
        g, w = got[name], want[name]
        if name in ("dbeta", "dg"):
            check(name, g, w, R.GDR)
        elif name == "dS0":
            check(name, g.flatten(2), w.flatten(2), R.GDR)
        else:
            check(name, g, w, R.GDR_BF16_DK if name == "dk" and dt != torch.float32 else R.GDR, dt)


SIZES = [(1, 1, 1, 64, 64), (2, 3, 1, 33, 40), (1, 2, 16, 128, 128), (2, 2, 17, 64, 64), (2, 1, 32, 64, 64), (1, 2, 33, 64, 64), (1, 1, 63, 16, 16),
         (2, 1, 64, 64, 64), (1, 3, 65, 64, 64), (1, 2, 128, 1, 1), (2, 2, 200, 40, 100), (1, 2, 130, 128, 64),
         (1, 2, 130, 64, 128), (1, 1, 300, 128, 128), (1, 2, 129, 65, 65), (3, 1, 90, 7, 3)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gdr_forward(dt, size):
    p, _ = inputs(*size, DT[dt])
    out, S = forward(p)
    check_forward(out, S, p)
    out2, S2 = forward(p)
    assert torch.equal(out, out2) and torch.equal(S, S2)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gdr_backward(dt, size):
    p, a = inputs(*size, DT[dt], 2)
    got = backward(p, a)
    check_backward(got, p, a)
    for name, t in backward(p, a).items():
        assert torch.equal(t, got[name]), name


@pytest.mark.parametrize("layout", ["blocks", "odd"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(2, 3, 1, 64, 64), (2, 2, 9, 20, 36), (2, 4, 131, 64, 64), (1, 2, 77, 100, 33)], ids=str)
@pytest.mark.parametrize("Hk", [1, None])
def test_gdr_layouts_and_shared_heads(layout, dt, size, Hk):
    p, a = inputs(*size, DT[dt], 3, Hk)
    out, S = forward(p, layout=layout)
    check_forward(out, S, p)
    dense = forward(p)
    assert torch.equal(out, dense[0]) and torch.equal(S, dense[1])
    got = backward(p, a, layout=layout)
    check_backward(got, p, a)
    for name, t in backward(p, a).items():
        assert torch.equal(t, got[name]), name


@pytest.mark.parametrize("T", [5, 70, 200])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gdr_lengths_and_rows_behind_them(T, dt):
    """Rows behind a sequence's end hold NaN and infinities, which must not be read; they come back as zeros."""
    n = torch.tensor([T, 0, 1, T - 1, T + 5, -3, T // 2], dtype=torch.int32)
    p, a = inputs(7, 2, T, 64, 48, DT[dt], 4)
    bad = ~SR.valid(n, 7, T)
    clean = {k: v.clone() for k, v in p.items()}, dict(a)
    for t, x in ((p["q"], math.nan), (p["k"], math.inf), (p["v"], math.nan), (a["dout"], -math.inf)):
        t[bad.expand(t.shape)] = x
    for t, x in ((p["beta"], math.nan), (p["g"], math.inf)):
        t[bad[..., 0].expand(t.shape)] = x
    out, S = forward(p, n)
    check_forward(out, S, clean[0], n)
    assert torch.equal(S[1].cpu(), p["S0"][1]) and torch.equal(S[5].cpu(), p["S0"][5])
    assert not out.cpu()[bad.expand(out.shape)].any()
    got = backward(p, a, n)
    a["dout"][bad.expand(a["dout"].shape)] = 0
    check_backward(got, clean[0], a, n)
    assert torch.equal(got["dS0"][1].cpu(), a["dS_final"][1])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gdr_long_sequences_in_segments(dt):
    """Few heads and many chunks: the scan goes by segments, whose last is short, and one sequence ends inside."""
    n = torch.tensor([2500, 1300], dtype=torch.int32)
    p, a = inputs(2, 1, 2500, 32, 24, DT[dt], 5)
    out, S = forward(p, n)
    check_forward(out, S, p, n)
    check_backward(backward(p, a, n), p, a, n)
    p, a = inputs(1, 2, 1100, 128, 72, DT[dt], 6, Hk=1)
    out, S = forward(p)
    check_forward(out, S, p)
    check_backward(backward(p, a), p, a)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gdr_continues_from_its_state(dt):
    """A prefill and steps of one and a few tokens, the state updated in place, make what one call makes."""
    p, _ = inputs(2, 3, 100, 64, 64, DT[dt], 7)
    cut = lambda a, b: {n: (t[:, :, a:b] if n != "S0" else t) for n, t in p.items()}  # noqa: E731
    S = p["S0"].cuda()
    outs, at = [], 0
    for n in (50, 1, 1, 5, 33, 10):
        q = cut(at, at + n)
        o, s = F.gdr_forward(*(q[x].cuda() for x in ("q", "k", "v", "beta", "g")), S, S_final=S)
        assert s is S
        outs.append(o)
        at += n
    check_forward(torch.cat(outs, 2), S, p)


def test_gdr_without_state():
    for T in (3, 100):
        p, a = inputs(1, 2, T, 64, 64, torch.float32, 8, S0=False)
        out, S = forward(p, want_state=False)
        assert S is None
        check("out", out, R.gdr_forward(**p)[0], R.GDR)
        a["dS_final"] = None
        check_backward(backward(p, a), p, a)


@pytest.mark.parametrize("T", [6, 150])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gdr_gates_at_their_ends(T, dt):
    """Gains of 0 and 1, decays of nothing and of everything (-inf, and what rounds to it), in one sequence."""
    p, a = inputs(1, 2, T, 64, 64, DT[dt], 9)
    p["beta"][:, :, ::3] = 0
    p["beta"][:, :, 1::5] = 1
    p["g"][:, 0] = 0
    p["g"][:, 1, T // 2] = -math.inf
    p["g"][:, 1, T // 3] = -3e38
    p["g"][:, 1, 2] = -90.0
    out, S = forward(p)
    check_forward(out, S, p)
    got = backward(p, a)
    check_backward(got, p, a)
    gone = p["g"] < -150  # e^g is 0 in fp32 (at -90 it is not)
    assert gone.any() and not got["dg"].cpu()[gone].any()


def test_gdr_reads_gates_of_every_size_to_fp32():
    """Decays of e^-1 and of 1 - 1e-6 beside one another: differences of a chunk's sums keep their precision."""
    p, a = inputs(1, 1, 128, 64, 64, torch.float32, 10)
    p["g"] = torch.where(torch.arange(128) % 7 == 0, torch.tensor(-1.0), torch.tensor(-1e-6)).expand(1, 1, 128).contiguous()
    out, S = forward(p)
    check_forward(out, S, p)
    check_backward(backward(p, a), p, a)


@pytest.mark.parametrize("T", [1, 80])
def test_gdr_nan_stays_in_its_head_and_behind_its_token(T):
    p, _ = inputs(1, 3, T, 64, 64, torch.bfloat16, 11)
    p["v"][0, 1, T // 2, 5] = math.nan
    out, S = forward(p)
    assert torch.isnan(S[0, 1, :, 5]).all() and torch.isnan(out[0, 1, T // 2, 5])
    assert not torch.isnan(S[0, ::2]).any() and not torch.isnan(out[0, ::2]).any()


def test_gdr_without_tokens():
    """No tokens, or none in any sequence: the states pass through."""
    p, a = inputs(2, 3, 0, 40, 64, torch.bfloat16, 27)
    out, S = F.gdr_forward(*(p[n].cuda() for n in ("q", "k", "v", "beta", "g")), p["S0"].cuda())
    assert out.shape == (2, 3, 0, 64) and torch.equal(S.cpu(), p["S0"])
    got = F.gdr_backward(*(p[n].cuda() for n in ("q", "k", "v", "beta", "g")), a["dout"].cuda(), p["S0"].cuda(), a["dS_final"].cuda())
    assert torch.equal(got["dS0"].cpu(), a["dS_final"]) and got["dq"].shape == (2, 3, 0, 40)
    p, a = inputs(2, 2, 100, 64, 64, torch.float32, 28, Hk=1)
    n = torch.zeros(2, dtype=torch.int32)
    out, S = forward(p, n)
    assert not out.any() and torch.equal(S.cpu(), p["S0"])
    got = backward(p, a, n)
    assert torch.equal(got["dS0"].cpu(), a["dS_final"])
    assert not any(got[x].any() for x in ("dq", "dk", "dv", "dbeta", "dg"))


def test_gdr_gains_of_every_size():
    """dbeta is formed from what has the gain as a factor: gains from 0 through 1e-30 and 1e-12 to 1, and below 0."""
    p, a = inputs(1, 2, 100, 64, 64, torch.float32, 29)
    p["beta"][0, 0] = torch.logspace(-38, 0, 100)
    p["beta"][0, 1, ::2] *= -1
    out, S = forward(p)
    check_forward(out, S, p)
    got = backward(p, a)
    check_backward(got, p, a)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    # each token's own: rows of dv carry their gain, however small
    for t in range(100):
        check(f"dv of token {t}", got["dv"][:, :1, t:t + 1], want["dv"][:, :1, t:t + 1], 4 * R.GDR)
        check(f"dbeta of token {t}", got["dbeta"][:, :1, t:t + 1, None], want["dbeta"][:, :1, t:t + 1, None], 40 * R.GDR)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gain", [1.0, 1.9])
def test_gdr_one_key_for_all_tokens(dt, gain):
    """Every token writes where the one before it wrote: the triangle is full, its inverse's signs alternate."""
    p, a = inputs(1, 2, 200, 64, 64, DT[dt], 30)
    p["k"] = torch.zeros_like(p["k"])
    p["k"][..., 5] = 1.0
    p["beta"] = torch.full_like(p["beta"], gain)
    p["g"] = torch.full_like(p["g"], -1e-3)
    out, S = forward(p)
    check_forward(out, S, p)
    check_backward(backward(p, a), p, a)


@pytest.mark.parametrize("T", [20, 70])
def test_gdr_strong_decays(T):
    """Decays that leave e^-6 of a state: dg is small beside the sums it comes from."""
    p, a = inputs(2, 2, T, 64, 64, torch.float32, 31)
    p["g"] = torch.full_like(p["g"], -6.0)
    out, S = forward(p)
    check_forward(out, S, p)
    got = backward(p, a)
    want = R.gdr_backward(p["q"], p["k"], p["v"], p["beta"], p["g"], a["dout"], p["S0"], a["dS_final"])
    terms = (want["dq"] * p["q"]).sum(-1).abs() + (want["dv"] * p["v"]).sum(-1).abs()
    off = (got["dg"].cpu().double() - want["dg"]).norm(dim=-1)
    assert (off <= R.GDR * terms.norm(dim=-1)).all()


def test_gdr_scale():
    p, a = inputs(1, 2, 70, 64, 64, torch.float32, 12)
    for scale in (1.0, 0.0, -2.5):
        out, S = forward(p, scale=scale)
        check_forward(out, S, p, scale=scale)
        check_backward(backward(p, a, scale=scale), p, a, scale=scale)


def test_gdr_broadcast_inputs():
    """One row read for many places: head and token strides of 0."""
    p, a = inputs(2, 4, 40, 32, 32, torch.float32, 13)
    for n in ("q", "k"):
        p[n] = p[n][:, :1].expand(2, 4, 40, 32)
    p["v"] = p["v"][:1].expand(2, 4, 40, 32)
    for n in ("beta", "g"):
        p[n] = p[n][:, :, :1].expand(2, 4, 40)
    dev = {"S0": p["S0"].cuda()}
    for n in ("q", "k", "v", "beta", "g"):
        dev[n] = torch.empty_strided(p[n].shape, p[n].stride(), dtype=p[n].dtype, device="cuda")
        at = tuple(slice(0, 1) if s == 0 else slice(None) for s in p[n].stride())
        dev[n][at] = p[n][at].cuda()
    args = [dev[n] for n in ("q", "k", "v", "beta", "g")]
    out, S = F.gdr_forward(*args, dev["S0"])
    check_forward(out, S, p)
    got = F.gdr_backward(*args, a["dout"].cuda(), dev["S0"], a["dS_final"].cuda())
    check_backward(got, p, a)


def test_gdr_writes_stay_inside():
    """Outputs as views into larger buffers: what lies around them keeps its bits."""
    for T, dv in ((3, 20), (70, 20), (70, 64)):
        p, a = inputs(1, 2, T, 24, dv, torch.bfloat16, 14)
        big = torch.full((1, 2, T + 4, dv + 6), 7.0, dtype=torch.bfloat16, device="cuda")
        state = torch.full((2, 2, 24, dv), 7.0, device="cuda")
        ws_n = F.falcon_gdr_workspace_bytes(F.make_gdr_dims(1, 2, T, 24, dv))
        ws = torch.full((ws_n + 512,), 0xff, dtype=torch.uint8, device="cuda")
        out, S = forward(p, out=big[:, :, 2:-2, 3:-3], S_final=state[1:], workspace=ws[:ws_n] if ws_n else None)
        check_forward(out, S, p)
        big[:, :, 2:-2, 3:-3] = 7.0
        assert (big == 7).all() and (state[0] == 7).all() and (ws[ws_n:] == 0xff).all()
        ws_n = F.falcon_gdr_workspace_bytes(F.make_gdr_dims(1, 2, T, 24, dv), True)
        ws = torch.full((ws_n + 512,), 0xff, dtype=torch.uint8, device="cuda")
        got = backward(p, a, dv=big[:, :, 2:-2, 3:-3], workspace=ws[:ws_n])
        check_backward(got, p, a)
        big[:, :, 2:-2, 3:-3] = 7.0
        assert (big == 7).all() and (ws[ws_n:] == 0xff).all()


def test_gdr_offsets_past_32_bits():
    B, T, d = 2, 70, 64
    far = 2 ** 31 + 64  # elements between the two sequences
    p, a = inputs(B, 1, T, d, d, torch.bfloat16, 15)
    buf = torch.empty(far + 3 * T * d, dtype=torch.bfloat16, device="cuda")
    view = lambda i: torch.as_strided(buf, (B, 1, T, d), (far, T * d, 3 * d, 1), i * d)  # noqa: E731
    q, k, v = (view(i).copy_(p[n]) for i, n in enumerate(("q", "k", "v")))
    out = torch.as_strided(torch.empty(far + T * d, dtype=torch.bfloat16, device="cuda"), (B, 1, T, d), (far, T * d, d, 1))
    beta, g, S0 = p["beta"].cuda(), p["g"].cuda(), p["S0"].cuda()
    _, S = F.gdr_forward(q, k, v, beta, g, S0, out=out)
    check_forward(out, S, p)
    got = F.gdr_backward(q, k, v, beta, g, a["dout"].cuda(), S0, a["dS_final"].cuda(), dv=out)
    check_backward(got, p, a)


def test_gdr_many_sequences():
    p, a = inputs(700, 3, 2, 16, 16, torch.bfloat16, 16)
    check_forward(*forward(p), p)
    p, a = inputs(300, 2, 40, 16, 16, torch.bfloat16, 17)
    check_forward(*forward(p), p)
    check_backward(backward(p, a), p, a)


# ---- the norm


def rms_inputs(B, T, d, dt, seed, residual=True):
    r = Draw(seed)
    x = r(B, T, d).to(dt)
    return x, (r(B, T, d) * torch.exp(r(B, T, 1))).to(dt) if residual else None, 1 + 0.3 * r(d)


def place_rows(layout, *tensors):
    if layout == "dense":
        return [t.cuda() for t in tensors]
    if layout == "odd":
        return [torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t) for t in tensors]
    out = []
    for t in tensors:  # tokens of every batch beside one another, with a gap behind each
        B, T, d = t.shape
        buf = torch.full((T, B, d + 16), 3.0, device="cuda").to(t.dtype)
        out.append(buf[:, :, :d].transpose(0, 1).copy_(t))
    return out


def check_norm(y, h, scales, x, w, residual, lengths=None, eps=1e-6):
    ry, rh = R.rms_forward(x, w, residual, eps=eps, lengths=lengths)
    d = x.shape[-1]
    assert torch.equal(h.cpu().view(rh.shape), rh) or residual is None
    y = y.cpu()
    if scales is None:
        bound = (R.half_step(x.dtype) + R.rms_room(d)) * ry.abs()
        assert ((y.double() - ry).abs() <= bound).all()
        return
    top = ry.abs().amax(-1)
    assert ((scales.cpu().double() - top / 448).abs() <= (R.rms_room(d) + 4 * R.U) * top / 448).all()
    # the value lies within half a step of the exact quotient, moved by the quotient's own error
    s = torch.where(top > 0, top / 448, 1.0)[..., None]
    quo = ry / s
    step = torch.exp2(torch.floor(torch.log2(quo.abs().clamp(min=2.0 ** -6))) - 3)
    room = 3 * (R.rms_room(d) + 4 * R.U) * quo.abs()
    assert ((y.double() - quo).abs() <= step / 2 + room).all()
    assert ((y.double() == R.e4m3(quo)).double().mean() > 0.999)


RMS_D = [1, 3, 8, 33, 64, 100, 255, 512, 513, 768, 1000, 1024, 1032, 2048, 4097, 8192, 8200, 12345, 16384]


@pytest.mark.parametrize("d", RMS_D)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("eight", [False, True])
def test_rms_forward(d, dt, eight):
    x, res, w = rms_inputs(2, 5, d, DT[dt], d)
    for r in (res, None):
        y, h, s = F.rmsnorm_forward(x.cuda(), w.cuda(), gpu(r), out_dtype=E4M3 if eight else None)
        assert y.dtype == (E4M3 if eight else x.dtype) and (s is not None) == eight
        check_norm(y, h, s, x, w, r)


@pytest.mark.parametrize("d", RMS_D)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rms_backward(d, dt):
    x, h, w = rms_inputs(2, 5, d, DT[dt], d + 1)
    dh = Draw(d)(2, 5, d).to(DT[dt])
    for extra in (dh, None):
        got = F.rmsnorm_backward(h.cuda(), x.cuda(), w.cuda(), gpu(extra))
        check_norm_backward(got, h, x, w, extra)


def check_norm_backward(got, h, dy, w, dh, lengths=None):
    (dx, dw), (ex, ew) = R.rms_backward(h, dy, w, dh, lengths=lengths)
    d = got["dx"].cpu().double()
    assert ((d - dx).abs() <= R.half_step(h.dtype) * dx.abs() + 1.01 * ex + 1e-30).all()
    if got["dweight"] is not None:
        assert ((got["dweight"].cpu().double() - dw).abs() <= ew + 1e-30).all()


@pytest.mark.parametrize("layout", ["dense", "odd", "gaps"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 768), (6, 37, 768), (5, 3, 96), (3, 50, 2048)], ids=str)
def test_rms_layouts_and_lengths(layout, dt, shape):
    B, T, d = shape
    x, res, w = rms_inputs(*shape, DT[dt], 3)
    dh = Draw(4)(*shape).to(DT[dt])
    n = torch.tensor([T, 0, T // 2, T + 3, -1, 1][:B], dtype=torch.int32)
    bad = (~SR.valid(n, B, T))[:, 0].expand(shape)
    clean = [t.clone() for t in (x, res, dh)]
    for t in (x, res, dh):
        t[bad] = math.nan
    xd, rd, hd, y, h, dx = place_rows(layout, x, res, dh, *(torch.full(shape, math.nan, dtype=DT[dt]) for _ in range(3)))
    got = F.rmsnorm_forward(xd, w.cuda(), rd, lengths=n.cuda(), y=y, h=h)
    assert got[0] is y and got[1] is h
    check_norm(y, h, None, clean[0], w, clean[1], n)
    y8, _, s = F.rmsnorm_forward(xd, w.cuda(), rd, lengths=n.cuda(), out_dtype=E4M3)
    check_norm(y8, h, s, clean[0], w, clean[1], n)
    got = F.rmsnorm_backward(rd, xd, w.cuda(), hd, lengths=n.cuda(), dx=dx)
    check_norm_backward(got, clean[1], clean[0], w, clean[2], n)


def test_rms_in_place_and_flat_tokens():
    x, res, w = rms_inputs(1, 9, 768, torch.bfloat16, 5)
    want = F.rmsnorm_forward(x.cuda(), w.cuda(), res.cuda())
    for own in ("x", "residual"):
        a, b = x.cuda()[0], res.cuda()[0]
        h = a if own == "x" else b
        y, got, _ = F.rmsnorm_forward(a, w.cuda(), b, h=h)
        assert got is h and torch.equal(h, want[1][0]) and torch.equal(y, want[0][0])
    dh = Draw(6)(9, 768).bfloat16().cuda()
    ref = F.rmsnorm_backward(want[1][0], x.cuda()[0], w.cuda(), dh)
    g = dh.clone()
    got = F.rmsnorm_backward(want[1][0], x.cuda()[0], w.cuda(), g, dx=g)
    assert got["dx"] is g and torch.equal(g, ref["dx"]) and torch.equal(got["dweight"], ref["dweight"])


def test_rms_optional_parameters():
    x, _, _ = rms_inputs(2, 7, 200, torch.float32, 7)
    y, h, s = F.rmsnorm_forward(x.cuda())
    check_norm(y, h, s, x, None, None)
    dy = Draw(8)(2, 7, 200)
    got = F.rmsnorm_backward(x.cuda(), dy.cuda(), want_params=False)
    assert got["dweight"] is None
    check_norm_backward(got, x, dy, None, None)


def test_rms_rows_of_zeros_nan_and_tiny_values():
    x = torch.zeros(1, 5, 256)
    x[0, 1, 3] = math.nan
    x[0, 2] = 1e-30
    x[0, 3] = 1.0
    y, _, s = F.rmsnorm_forward(x.cuda(), None, out_dtype=E4M3)
    assert s[0, 0] == 0 and not y[0, 0].float().any()
    assert torch.isnan(s[0, 1]) and torch.isnan(y[0, 1].float()).all()
    assert (y[0, 2].float() == 448).all() and (y[0, 3].float() == 448).all()
    w = torch.full((256,), 1e-38)
    w[1:] = 5e-39
    y, _, s = F.rmsnorm_forward(x.cuda(), w.cuda(), out_dtype=E4M3)  # scales below the least normal number
    assert abs(y[0, 3, 0].float().item() - 448) <= 16 and abs(y[0, 3, 1].float().item() - 224) <= 8
    y, _, _ = F.rmsnorm_forward(x.cuda(), None)
    assert not y[0, 0].any() and torch.isnan(y[0, 1]).all() and not torch.isnan(y[0, 2:]).any()


def test_rms_many_tokens():
    x, h, w = rms_inputs(3, 3001, 64, torch.bfloat16, 9)
    y, hh, _ = F.rmsnorm_forward(x.cuda(), w.cuda(), h.cuda())
    check_norm(y, hh, None, x, w, h)
    got = F.rmsnorm_backward(h.cuda(), x.cuda(), w.cuda(), None)
    check_norm_backward(got, h, x, w, None)
    assert torch.equal(got["dweight"], F.rmsnorm_backward(h.cuda(), x.cuda(), w.cuda(), None)["dweight"])


def test_rms_offsets_past_32_bits():
    far = 2 ** 31 + 128
    x, res, w = rms_inputs(2, 3, 100, torch.bfloat16, 10)
    buf = torch.empty(far + 1000, dtype=torch.bfloat16, device="cuda")
    v = [torch.as_strided(buf, (2, 3, 100), (far, 100, 1), 300 * i) for i in range(3)]
    v[0].copy_(x), v[1].copy_(res)
    y, h, _ = F.rmsnorm_forward(v[0], w.cuda(), v[1], y=v[2])
    check_norm(y, h, None, x, w, res)
    got = F.rmsnorm_backward(v[1], v[0], w.cuda(), dx=v[2])
    check_norm_backward(got, res, x, w, None)


# ---- streams, captures, threads, and a block of them together


def block(x, res, p, weights, S0, eight=False):
    """Pre-norm, one projection, delta rule, the read's norm with its gate, the projection back."""
    wn, win, wg, wout = weights
    B, T, D = x.shape
    H, dk = S0.shape[1], S0.shape[2]
    y, h, _ = F.rmsnorm_forward(x, wn, res)
    qkvz = y @ win
    heads = [t.unflatten(2, (H, dk)).transpose(1, 2) for t in qkvz.split(H * dk, 2)]
    out, S = F.gdr_forward(*heads[:3], p["beta"], p["g"], S0)
    o = F.groupnorm_forward(out, wg, None, heads[3], act="silu")
    return o.transpose(1, 2).reshape(B, T, H * dk) @ wout, h, out, S, heads, o


def test_block_forward_and_back():
    """The operators in a row, as a layer runs them, against the same layer in double with autograd on the CPU."""
    B, T, H, dk = 2, 90, 2, 32
    D = H * dk
    r = Draw(20)
    x, res = r(B, T, D), r(B, T, D)
    win, wout, wn, wg = r(D, 4 * D) / D ** 0.5, r(D, D) / D ** 0.5, 1 + 0.2 * r(D), 1 + 0.2 * r(H, dk)
    # keys of about unit length come from the projection scaled down
    win[:, D:2 * D] /= dk ** 0.5
    beta, g, S0 = torch.sigmoid(r(B, H, T)), -torch.exp(r(B, H, T) - 3), r(B, H, dk, dk) / dk ** 0.5
    dy, dh = r(B, T, D), r(B, T, D)
    dev = lambda t: t.cuda()  # noqa: E731
    prec = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        p = dict(beta=dev(beta), g=dev(g))
        xd, rd, wnd, wind, wgd, woutd, Sd = map(dev, (x, res, wn, win, wg, wout, S0))
        y, h, out, S, heads, o = block(xd, rd, p, (wnd, wind, wgd, woutd), Sd)
        do = (dev(dy) @ woutd.T).unflatten(2, (H, dk)).transpose(1, 2)
        dn = F.groupnorm_backward(out, do, wgd, None, heads[3], act="silu")
        dqkvz = torch.empty(B, T, 4 * D, device="cuda")
        dheads = [t.unflatten(2, (H, dk)).transpose(1, 2) for t in dqkvz.split(D, 2)]
        dheads[3].copy_(dn["dz"])
        dd = F.gdr_backward(*heads[:3], p["beta"], p["g"], dn["dx"], Sd, dq=dheads[0], dk=dheads[1], dv=dheads[2])
        dr = F.rmsnorm_backward(h, dqkvz @ wind.T, wnd, dev(dh))
    finally:
        torch.backends.cuda.matmul.allow_tf32 = prec
    leaf = {n: t.double().requires_grad_() for n, t in dict(x=x, res=res, wn=wn, win=win, wg=wg, wout=wout, beta=beta, g=g,
                                                            S0=S0).items()}
    hc = leaf["x"] + leaf["res"]
    yc = hc / torch.sqrt(hc.square().mean(-1, keepdim=True) + 1e-6) * leaf["wn"]
    q, k, v, z = (t.unflatten(2, (H, dk)).transpose(1, 2) for t in (yc @ leaf["win"]).split(D, 2))
    Sc, reads = leaf["S0"], []
    for t in range(T):
        kept = leaf["g"][:, :, t, None, None].exp() * Sc
        err = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", kept, k[:, :, t])
        Sc = kept + k[:, :, t, :, None] * (leaf["beta"][:, :, t, None] * err)[:, :, None]
        reads.append(dk ** -0.5 * torch.einsum("bhkv,bhk->bhv", Sc, q[:, :, t]))
    oc = torch.stack(reads, 2)
    oc = oc - oc.mean(-1, keepdim=True)
    oc = oc / torch.sqrt(oc.square().mean(-1, keepdim=True) + 1e-5) * leaf["wg"][:, None] * torch.nn.functional.silu(z)
    final = oc.transpose(1, 2).reshape(B, T, D) @ leaf["wout"]
    ((final * dy.double()).sum() + (hc * dh.double()).sum()).backward()
    # each operator's own bound, times the products and norms between: the read's norm divides by its deviation
    for name, got, want in (("y", y, final.detach()), ("S", S.flatten(2), Sc.detach().flatten(2)), ("dx", dr["dx"], leaf["x"].grad),
                            ("dwn", dr["dweight"], leaf["wn"].grad), ("dbeta", dd["dbeta"], leaf["beta"].grad),
                            ("dg", dd["dg"], leaf["g"].grad), ("dS0", dd["dS0"].flatten(2), leaf["S0"].grad.flatten(2)),
                            ("dwg", dn["dweight"], leaf["wg"].grad)):
        check(name, got, want, 10 * R.GDR)
    assert torch.equal(leaf["x"].grad, leaf["res"].grad)


def test_captured_calls_replay_on_new_inputs():
    B, H, T, d = 2, 3, 150, 64
    p, a = inputs(B, H, T, d, d, torch.bfloat16, 21)
    p2, a2 = inputs(B, H, T, d, d, torch.bfloat16, 22)
    x, res, w = rms_inputs(B, T, 256, torch.bfloat16, 23)
    names = ("q", "k", "v", "beta", "g", "S0")
    dev = {n: p[n].cuda() for n in names}
    da = {n: t.cuda() for n, t in a.items()}
    xd, rd, wd = x.cuda(), res.cuda(), w.cuda()

    def once():
        out, S = F.gdr_forward(*(dev[n] for n in names))
        one, S1 = F.gdr_forward(*(dev[n][:, :, :1] for n in names[:5]), S)
        g = F.gdr_backward(*(dev[n] for n in names[:5]), da["dout"], dev["S0"], da["dS_final"])
        y, h, s = F.rmsnorm_forward(xd, wd, rd, out_dtype=E4M3)
        b = F.rmsnorm_backward(h, xd, wd, rd)
        return [out, S, one, S1, *g.values(), y.view(torch.uint8), h, s, *b.values()]

    once()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, results = [], []
    for _ in range(2):  # two graphs with buffers of their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            results.append(once())
        graphs.append(g)
    for q, b in ((p, a), (p2, a2)):
        for n in names:
            dev[n].copy_(q[n])
        for n in da:
            da[n].copy_(b[n])
        want = [t.clone() for t in once()]
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for res_ in results:
            for u, v in zip(res_, want):
                assert torch.equal(u, v)


def test_side_streams_at_the_same_time():
    p, a = inputs(2, 2, 300, 64, 64, torch.bfloat16, 24)
    want = [t.clone() for t in backward(p, a).values()]
    dev = {n: t.cuda() for n, t in p.items()}
    da = {n: t.cuda() for n, t in a.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for s in streams:
        got.append(F.gdr_backward(*(dev[n] for n in ("q", "k", "v", "beta", "g")), da["dout"], dev["S0"], da["dS_final"],
                                  stream=s))
    torch.cuda.synchronize()
    for g in got:
        for u, v in zip(g.values(), want):
            assert torch.equal(u, v)


PENDING = 40_000_000  # cycles of a kernel that does nothing, some 20 ms


def test_memory_belongs_to_the_given_stream():
    """The current stream allocates and writes while a call on another stream still waits: what the call allocated, its
    workspace too, is not among it."""
    p, a = inputs(2, 2, 300, 64, 64, torch.bfloat16, 27)
    dev, da = ({n: t.cuda() for n, t in x.items()} for x in (p, a))
    ok = [dev[n] for n in ("q", "k", "v", "beta", "g")]
    x, w = torch.randn(2000, 200, device="cuda"), torch.randn(200, device="cuda")

    def calls(stream):
        out = [*F.gdr_forward(*ok, dev["S0"], stream=stream)]
        out += F.gdr_backward(*ok, da["dout"], dev["S0"], da["dS_final"], stream=stream).values()
        out += F.rmsnorm_forward(x, w, x, out_dtype=E4M3, stream=stream)
        return out + [*F.rmsnorm_backward(x, x, w, x, stream=stream).values()]

    want = calls(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):  # the second time from memory that the first gave back
        with torch.cuda.stream(side):
            torch.cuda._sleep(PENDING)
        got = calls(side)
        over = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in (1 << k for k in range(9, 25)) for _ in range(4)]
        torch.cuda.synchronize()
        for u, v in zip(got, want):
            assert torch.equal(u.float(), v.float())
        del got, over


def test_two_host_threads():
    p, _ = inputs(2, 2, 200, 64, 64, torch.float32, 25)
    want = forward(p)
    failures = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out, S = forward(p)
                    torch.cuda.current_stream().synchronize()
                    assert torch.equal(out, want[0]) and torch.equal(S, want[1])
        except Exception as e:  # noqa: BLE001
            failures.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failures, failures


def test_wrappers_refuse():
    p, a = inputs(1, 2, 40, 16, 16, torch.bfloat16, 26)
    d = {n: t.cuda() for n, t in p.items()}
    ok = [d[n] for n in ("q", "k", "v", "beta", "g")]

    def swapped(i, t):
        return [t if j == i else x for j, x in enumerate(ok)]

    for args in (swapped(0, d["q"].half()), swapped(1, d["k"].float()), swapped(1, d["k"][:, :, :10]),
                 swapped(2, d["v"].transpose(2, 3)), swapped(3, d["beta"].bfloat16()), swapped(4, d["g"][:, :1]),
                 swapped(2, d["v"].cpu()), swapped(2, d["v"][0])):
        with pytest.raises(ValueError):
            F.gdr_forward(*args)
    with pytest.raises(ValueError):
        F.gdr_forward(*ok, d["S0"].double())
    with pytest.raises(ValueError):
        F.gdr_forward(*ok, lengths=torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(F.FalconError):
        F.gdr_forward(*ok, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(F.FalconError):
        F.gdr_forward(*ok, scale=math.inf)
    for args in (swapped(2, d["v"][..., :0]), [t[..., :0] if t.dim() == 4 else t for t in ok]):
        with pytest.raises(ValueError, match="channels"):
            F.gdr_forward(*args)
    three = torch.zeros(1, 3, 40, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="divide"):
        F.gdr_forward(d["q"], d["k"], three, ok[3], ok[4])
    x = torch.zeros(2, 4, 32, device="cuda")
    for kw in (dict(residual=x.bfloat16()), dict(residual=x[:, :2]), dict(h=x.clone()), dict(y=x.half()), dict(scales=x[..., 0].clone()),
               dict(weight=torch.zeros(31, device="cuda")), dict(y=x.clone(), out_dtype=E4M3), dict(out_dtype=torch.int8)):
        with pytest.raises(ValueError):
            F.rmsnorm_forward(x, **kw)
    with pytest.raises(F.FalconError):
        F.rmsnorm_forward(x, eps=0.0)
    with pytest.raises(F.FalconError):
        F.rmsnorm_forward(x, y=x)
