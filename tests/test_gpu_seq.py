"""GPU parity of the gated linear recurrence and the head norm against their 64-bit references, elementwise,
within the rounding bounds that the references derive (oracle/seq_ref.py)."""

import math

import pytest
import torch

from oracle import seq_ref as R
from weight_linear_attention_gb300 import falcon as F

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
GATES = ["decay", "sigmoid", "mix"]
ACTS = ["none", "silu", "gelu", "sigmoid"]


def _close(name, got, ref, bound):
    ok, share = R.close(got, ref, bound)
    print(f"PARITY {name}: {share:.3f} of the bound")
    assert ok, f"{name}: {share:.3f} of the bound"


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def __call__(self, *shape):
        return torch.randn(*shape, generator=self.g)


def place(layout, *tensors):
    """CPU tensors [B,H,T,d] on the GPU in a layout: dense, the projection's ("bthd"), or column blocks of one
    [B,T,n,H,d] buffer ("blocks"), or one element off every vector boundary ("odd")."""
    B, H, T, d = tensors[0].shape
    dt = tensors[0].dtype
    if layout == "dense":
        return [t.cuda() for t in tensors]
    if layout == "odd":
        out = []
        for t in tensors:
            buf = torch.empty(t.numel() + 1, dtype=dt, device="cuda")[1:].view(B, H, T, d)
            out.append(buf.copy_(t))
        return out
    n = 1 if layout == "bthd" else len(tensors)
    bufs = [torch.empty(B, T, n, H, d, dtype=dt, device="cuda") for _ in range(len(tensors) // n)]
    out = []
    for i, t in enumerate(tensors):
        v = bufs[i if n == 1 else 0][:, :, 0 if n == 1 else i].transpose(1, 2)
        out.append(v.copy_(t))
    return out


def poison(layout, n, shape, dt):
    """Uninitialised outputs stand out: filled with NaN."""
    return place(layout, *[torch.full(shape, math.nan).to(dt) for _ in range(n)])


def glr_inputs(gate, shape, dt, seed, h0=True):
    B, H, T, d = shape
    r = Draw(seed)
    x = r(*shape).to(dt)
    g = (-torch.exp(r(*shape) - 2) if gate == "decay" else r(*shape) + 2).to(dt)
    return x, g, (r(B, H, d) if h0 else None)


def gpu(t):
    return None if t is None else t.cuda()


def run_fwd(gate, x, g, h0, lengths, layout="dense", **kw):
    xd, gd = place(layout, x, g)
    out, = poison(layout if layout != "blocks" else "bthd", 1, x.shape, x.dtype)
    return F.glr_forward(gate, xd, gd, gpu(h0), lengths=gpu(lengths), out=out, **kw)


SHAPES = [(2, 3, 1, 64), (1, 2, 4, 16), (2, 1, 5, 64), (1, 1, 127, 64), (1, 2, 128, 64), (2, 1, 129, 32),
          (1, 1, 1023, 128), (2, 2, 2500, 64), (1, 1, 3001, 33), (3, 1, 300, 1), (1, 3, 260, 40), (1, 1, 0, 8)]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_glr_forward(gate, dt, shape):
    x, g, h0 = glr_inputs(gate, shape, DT[dt], 1)
    out, h = run_fwd(gate, x, g, h0, None)
    (ro, rh), (eo, eh) = R.glr_forward(gate, x, g, h0)
    _close("out", out, ro, eo)
    _close("h_final", h, rh, eh)
    out2, h2 = run_fwd(gate, x, g, h0, None)
    assert torch.equal(out, out2) and torch.equal(h, h2)


@pytest.mark.parametrize("layout", ["bthd", "blocks", "odd"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(2, 3, 1, 64), (2, 3, 259, 64), (3, 2, 50, 20), (2, 5, 4, 7)], ids=str)
def test_glr_layouts_give_the_same_bits(layout, dt, shape):
    x, g, h0 = glr_inputs("mix", shape, DT[dt], 2)
    out, h = run_fwd("mix", x, g, h0, None)
    out2, h2 = run_fwd("mix", x, g, h0, None, layout)
    (ro, rh), (eo, eh) = R.glr_forward("mix", x, g, h0)
    for o, s in ((out, h), (out2, h2)):
        _close("out", o, ro, eo)
        _close("h_final", s, rh, eh)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T", [3, 300, 2300])
def test_glr_ragged_lengths_and_rows_behind_them(gate, T):
    """Rows behind a sequence's end hold NaN and infinities, which must not be read; they come back as zeros."""
    n = torch.tensor([T, 0, 1, T - 1, T + 5, -3, T // 2], dtype=torch.int32)
    shape = (7, 2, T, 64)
    x, g, h0 = glr_inputs(gate, shape, torch.bfloat16, 3)
    bad = ~R.valid(n, 7, T).expand(shape)
    x[bad], g[bad] = math.nan, math.inf
    out, h = run_fwd(gate, x, g, h0, n, "bthd")
    (ro, rh), (eo, eh) = R.glr_forward(gate, x, g, h0, n)
    _close("out", out, ro, eo)
    _close("h_final", h, rh, eh)
    assert torch.equal(h[1].cpu(), h0[1]) and torch.equal(h[5].cpu(), h0[5])


def test_glr_without_state_and_in_place():
    x, g, h0 = glr_inputs("sigmoid", (2, 2, 300, 64), torch.float32, 4)
    out, h = run_fwd("sigmoid", x, g, None, None, want_state=False)
    assert h is None
    (ro, _), (eo, _) = R.glr_forward("sigmoid", x, g)
    _close("out", out, ro, eo)
    for T in (1, 300):
        s = h0.cuda()
        _, want = run_fwd("sigmoid", x[:, :, :T].contiguous(), g[:, :, :T].contiguous(), h0, None)
        _, got = F.glr_forward("sigmoid", x[:, :, :T].cuda(), g[:, :, :T].cuda(), s, h_final=s)
        assert got is s and torch.equal(s, want)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_extreme_gates(gate, dt):
    """-inf forgets everything before a token, +inf and large logits keep it, 0 decays by nothing."""
    shape = (1, 2, 400, 64)
    x, g, h0 = glr_inputs(gate, shape, DT[dt], 5)
    inf = math.inf
    for t, v in ((0, -inf), (7, -100.0), (8, 0.0), (130, -inf), (131, -inf), (200, -30.0), (399, -1e-3)):
        g[:, :, t] = v
    if gate != "decay":
        for t, v in ((20, inf), (21, 100.0), (22, 30.0), (256, inf)):
            g[:, :, t] = v
    out, h = run_fwd(gate, x, g, h0, None)
    (ro, rh), (eo, eh) = R.glr_forward(gate, x, g, h0)
    _close("out", out, ro, eo)
    _close("h_final", h, rh, eh)
    dout = Draw(6)(*shape).to(DT[dt])
    stored = out.cpu()
    got = F.glr_backward(gate, x.cuda(), g.cuda(), out, dout.cuda(), h0.cuda())
    ref, e = R.glr_backward(gate, x, g, stored, dout, h0)
    for k, r, b in zip(("dx", "dg", "dh0"), ref, e):
        _close(k, got[k], r, b)


def test_glr_nan_stays_in_its_channel_and_behind_its_token():
    x, g, h0 = glr_inputs("mix", (1, 1, 700, 64), torch.float32, 7)
    x[0, 0, 333, 5] = math.nan
    out, h = run_fwd("mix", x, g, h0, None)
    nan = torch.zeros(700, 64, dtype=torch.bool)
    nan[333:, 5] = True
    assert torch.equal(out[0, 0].isnan().cpu(), nan)
    assert h.isnan().sum() == 1


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_glr_steps_continue_a_prefill(dt):
    """A prefill and single tokens from its state: each within the bounds of one call over all tokens."""
    x, g, h0 = glr_inputs("mix", (3, 4, 150, 64), DT[dt], 8)
    (ro, rh), (eo, eh) = R.glr_forward("mix", x, g, h0)
    xd, gd = x.cuda(), g.cuda()
    out, s = F.glr_forward("mix", xd[:, :, :140], gd[:, :, :140], h0.cuda())
    outs = [out]
    for t in range(140, 150):
        o, s = F.glr_forward("mix", xd[:, :, t:t + 1], gd[:, :, t:t + 1], s, h_final=s)
        outs.append(o)
    _close("out", torch.cat(outs, 2), ro, eo)
    _close("h_final", s, rh, eh)


BWD_SHAPES = [(2, 3, 1, 64), (2, 1, 5, 64), (1, 2, 128, 64), (2, 1, 129, 32), (1, 1, 1025, 128), (2, 2, 2500, 64),
              (1, 1, 1500, 33), (1, 3, 260, 40), (1, 1, 0, 8)]


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", BWD_SHAPES, ids=str)
def test_glr_backward(gate, dt, shape):
    x, g, h0 = glr_inputs(gate, shape, DT[dt], 10)
    r = Draw(11)
    dout, dh = r(*shape).to(DT[dt]), r(shape[0], shape[1], shape[3])
    out = R.glr_forward(gate, x, g, h0)[0][0].to(DT[dt])
    args = (x.cuda(), g.cuda(), out.cuda(), dout.cuda(), h0.cuda(), dh.cuda())
    dx, dg = poison("dense", 2, shape, DT[dt])
    got = F.glr_backward(gate, *args, dx=dx, dg=dg)
    ref, e = R.glr_backward(gate, x, g, out, dout, h0, dh)
    for k, v, b in zip(("dx", "dg", "dh0"), ref, e):
        _close(k, got[k], v, b)
    again = F.glr_backward(gate, *args)
    for k in got:
        assert torch.equal(got[k], again[k])


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("T", [2, 300, 2300])
def test_glr_backward_ragged_into_one_buffer(gate, T):
    """Gradients written as column blocks of one buffer (one projection's gradient); padding is not read and its
    gradients are zero; no initial state, no final adjoint."""
    n = torch.tensor([T, 0, 1, T - 1, T + 9, T // 3], dtype=torch.int32)
    shape = (6, 3, T, 64)
    x, g, _ = glr_inputs(gate, shape, torch.bfloat16, 12)
    dout = Draw(13)(*shape).to(torch.bfloat16)
    out = R.glr_forward(gate, x, g, None, n)[0][0].to(torch.bfloat16)
    bad = ~R.valid(n, 6, T).expand(shape)
    for v in (x, g, out, dout):
        v[bad] = math.nan
    xd, gd, od, dd = place("blocks", x, g, out, dout)
    dx, dg = poison("blocks", 2, shape, torch.bfloat16)
    got = F.glr_backward(gate, xd, gd, od, dd, lengths=n.cuda(), dx=dx, dg=dg)
    ref, e = R.glr_backward(gate, x, g, out, dout, None, None, n)
    for k, v, b in zip(("dx", "dg", "dh0"), ref, e):
        _close(k, got[k], v, b)


def test_glr_backward_raw_call_without_optional_buffers():
    """x is not read unless the gate mixes; dh0 may be left out."""
    shape = (2, 2, 200, 64)
    x, g, h0 = glr_inputs("decay", shape, torch.float32, 14)
    dout = Draw(15)(*shape)
    out = R.glr_forward("decay", x, g, h0)[0][0].float()
    gd, od, dd, hd = (t.cuda() for t in (g, out, dout, h0))
    dx, dg = torch.empty_like(gd), torch.empty_like(gd)
    dims = F.make_seq_dims(*shape, dtype=F.FALCON_F32)
    assert F.falcon_glr_bwd(0, None, gd, od, hd, None, dd, None, dx, dg, None, dims) == F.FALCON_OK
    ref, e = R.glr_backward("decay", x, g, out, dout, h0)
    _close("dx", dx, ref[0], e[0])
    _close("dg", dg, ref[1], e[1])


def test_glr_broadcast_gate():
    """One gate row for every head and token (strides 0): the gradient is that of every place."""
    shape = (2, 3, 300, 64)
    x, _, h0 = glr_inputs("sigmoid", shape, torch.float32, 16)
    g = Draw(17)(2, 1, 1, 64).expand(shape)
    dout = Draw(18)(*shape)
    gd = g[:, :1, :1].contiguous().cuda().expand(shape)
    out, h = F.glr_forward("sigmoid", x.cuda(), gd, h0.cuda())
    (ro, rh), (eo, eh) = R.glr_forward("sigmoid", x, g, h0)
    _close("out", out, ro, eo)
    got = F.glr_backward("sigmoid", x.cuda(), gd, out, dout.cuda(), h0.cuda())
    ref, e = R.glr_backward("sigmoid", x, g, out.cpu(), dout, h0)
    _close("dg", got["dg"], ref[1], e[1])


def test_glr_many_sequences_and_many_channels():
    """More sequences than fit the GPU at once, and one sequence of very many channels."""
    for shape in ((700, 2, 130, 64), (1, 1, 300, 20000)):
        x, g, h0 = glr_inputs("mix", shape, torch.bfloat16, 19)
        out, h = run_fwd("mix", x, g, h0, None)
        (ro, rh), (eo, eh) = R.glr_forward("mix", x, g, h0)
        _close("out", out, ro, eo)
        _close("h_final", h, rh, eh)


def _big(rows, d):
    """[2,1,rows,d] bf16 whose second sequence starts more than 2^31 elements behind the first."""
    far = (1 << 31) + 64
    buf = torch.empty(far + rows * d, dtype=torch.bfloat16, device="cuda")
    return buf.as_strided((2, 1, rows, d), (far, far, d, 1))


def test_offsets_past_32_bits():
    shape = (2, 1, 40, 64)
    x, g, h0 = glr_inputs("mix", shape, torch.bfloat16, 20)
    xd, gd, od = _big(40, 64), _big(40, 64), _big(40, 64)
    xd.copy_(x), gd.copy_(g)
    out, h = F.glr_forward("mix", xd, gd, h0.cuda(), out=od)
    (ro, rh), (eo, eh) = R.glr_forward("mix", x, g, h0)
    _close("out", out, ro, eo)
    y = F.groupnorm_forward(xd, z=gd, act="silu", y=od)
    _close("y", y, *R.gn_forward(x, z=g, name="silu"))
    got = F.groupnorm_backward(xd, gd, act="none", dx=od)
    ref, e = R.gn_backward(x, g)
    for k in ("dx", "dweight", "dbias"):
        _close(k, got[k], ref[k], e[k])


def gn_inputs(shape, dt, seed, gated):
    B, H, T, d = shape
    r = Draw(seed)
    x = (r(*shape) * torch.exp(r(1, H, 1, 1)) + 0.5 * r(1, H, 1, d)).to(dt)
    z = r(*shape).to(dt) if gated else None
    return x, z, 1 + 0.3 * r(H, d), 0.3 * r(H, d), r(*shape).to(dt)


GN_D = [1, 2, 7, 16, 33, 40, 64, 72, 100, 128, 200, 256, 257, 384, 512, 513, 768, 1000, 1023, 1024]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", GN_D)
def test_groupnorm(act, gated, dt, d):
    shape = (2, 3, 11, d)
    x, z, w, b, dy = gn_inputs(shape, DT[dt], 30 + d, gated)
    eps = 1e-5 if d > 2 else 0.1  # rows of one or two channels have little variance: eps decides
    xd, dd, wd, bd, zd = x.cuda(), dy.cuda(), w.cuda(), b.cuda(), gpu(z)
    y, = poison("bthd", 1, shape, DT[dt])
    y = F.groupnorm_forward(xd, wd, bd, zd, act=act, eps=eps, y=y)
    _close("y", y, *R.gn_forward(x, w, b, z, act, eps))
    dx, dz = poison("dense", 2, shape, DT[dt])
    got = F.groupnorm_backward(xd, dd, wd, bd, zd, act=act, eps=eps, dx=dx, dz=dz if gated else None)
    ref, e = R.gn_backward(x, dy, w, b, z, act, eps)
    for k in ref:
        _close(k, got[k], ref[k], e[k])
    again = F.groupnorm_backward(xd, dd, wd, bd, zd, act=act, eps=eps)
    for k in ref:
        assert torch.equal(got[k], again[k])


@pytest.mark.parametrize("layout", ["dense", "bthd", "blocks", "odd"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 64), (5, 3, 1, 64), (2, 12, 301, 64), (3, 2, 7, 48), (1, 1, 2000, 768)],
                         ids=str)
@pytest.mark.parametrize("ragged", [False, True])
def test_groupnorm_layouts_and_lengths(layout, shape, ragged):
    B, H, T, d = shape
    x, z, w, b, dy = gn_inputs(shape, torch.bfloat16, 50, True)
    n = torch.tensor([(T * (B - i)) // B if i != 1 else 0 for i in range(B)], dtype=torch.int32) if ragged else None
    if ragged:
        n[-1] += 1
        bad = ~R.valid(n, B, T).expand(shape)
        for v in (x, z, dy):
            v[bad] = math.nan
    xd, zd, dd = place(layout, x, z, dy)
    wd, bd = w.cuda(), b.cuda()
    nd = gpu(n)
    y, dx, dz = poison(layout, 3, shape, torch.bfloat16)
    y = F.groupnorm_forward(xd, wd, bd, zd, act="silu", lengths=nd, y=y)
    _close("y", y, *R.gn_forward(x, w, b, z, "silu", 1e-5, n))
    got = F.groupnorm_backward(xd, dd, wd, bd, zd, act="silu", lengths=nd, dx=dx, dz=dz)
    ref, e = R.gn_backward(x, dy, w, b, z, "silu", 1e-5, n)
    for k in ref:
        _close(k, got[k], ref[k], e[k])


# a width for every split of a row over lanes, and its neighbour that leaves lanes idle
GN_LANES = [8, 15, 20, 24, 31, 32, 47, 48, 49, 60, 63, 80, 96, 99, 127, 129, 160, 255, 300, 520, 700]


@pytest.mark.parametrize("layout", ["dense", "bthd", "odd"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", GN_LANES)
def test_groupnorm_lanes(layout, dt, d):
    shape = (3, 3, 157, d)
    x, z, w, b, dy = gn_inputs(shape, DT[dt], 70 + d, True)
    n = torch.tensor([157, 0, 80], dtype=torch.int32)
    xd, zd, dd = place(layout, x, z, dy)
    wd, bd = w.cuda(), b.cuda()
    y, dx, dz = poison(layout, 3, shape, DT[dt])
    y = F.groupnorm_forward(xd, wd, bd, zd, act="silu", lengths=n.cuda(), y=y)
    _close("y", y, *R.gn_forward(x, w, b, z, "silu", 1e-5, n))
    got = F.groupnorm_backward(xd, dd, wd, bd, zd, act="silu", lengths=n.cuda(), dx=dx, dz=dz)
    ref, e = R.gn_backward(x, dy, w, b, z, "silu", 1e-5, n)
    for k in ref:
        _close(k, got[k], ref[k], e[k])


def test_groupnorm_optional_parameters():
    x, z, w, b, dy = gn_inputs((2, 2, 9, 64), torch.float32, 60, True)
    xd, dd = x.cuda(), dy.cuda()
    y = F.groupnorm_forward(xd)
    assert y.transpose(1, 2).is_contiguous()
    _close("y", y, *R.gn_forward(x))
    _close("y", F.groupnorm_forward(xd, w.cuda()), *R.gn_forward(x, w))
    _close("y", F.groupnorm_forward(xd, None, b.cuda()), *R.gn_forward(x, None, b))
    got = F.groupnorm_backward(xd, dd, want_params=False)
    assert got["dweight"] is None and got["dbias"] is None and got["dz"] is None
    ref, e = R.gn_backward(x, dy)
    _close("dx", got["dx"], ref["dx"], e["dx"])
    only = F.groupnorm_backward(xd, dd, want_params=False, dbias=torch.empty(2, 64, device="cuda"))
    _close("dbias", only["dbias"], ref["dbias"], e["dbias"])
    empty = F.groupnorm_backward(xd[:, :, :0], dd[:, :, :0])
    assert not empty["dweight"].any() and not empty["dbias"].any()


def test_groupnorm_rows_without_variance():
    """Equal channels: the centred row is zero (its mean is exact here), y is the bias."""
    x = torch.full((1, 2, 5, 64), 3.0)
    b = Draw(61)(2, 64)
    y = F.groupnorm_forward(x.cuda(), None, b.cuda())
    assert torch.equal(y.cpu(), b[None, :, None].expand(1, 2, 5, 64))
    x[0, 0, 2, 3] = math.inf
    y = F.groupnorm_forward(x.cuda(), None, b.cuda()).cpu()
    assert y[0, 0, 2].isnan().all() and not y[0, 1].isnan().any() and not y[0, 0, 3].isnan().any()


def test_groupnorm_many_rows():
    x, z, w, b, dy = gn_inputs((3, 7, 5003, 64), torch.bfloat16, 62, True)
    args = [t.cuda() for t in (x, dy, w, b, z)]
    _close("y", F.groupnorm_forward(args[0], args[2], args[3], args[4], act="silu"), *R.gn_forward(x, w, b, z, "silu"))
    got = F.groupnorm_backward(*args, act="silu")
    ref, e = R.gn_backward(x, dy, w, b, z, "silu")
    for k in ref:
        _close(k, got[k], ref[k], e[k])


def test_side_stream_and_graph_replay():
    """Every call captured into one graph (a mixer's forward and backward) and replayed on new inputs; the same
    calls on two streams at once."""
    shape, dt = (2, 3, 1500, 64), torch.bfloat16
    w, b = Draw(70)(3, 64).cuda(), Draw(71)(3, 64).cuda()

    def inputs(seed):
        x, g, h0 = glr_inputs("mix", shape, dt, seed)
        r = Draw(seed + 100)
        return [t.cuda() for t in (x, g, h0, r(*shape).to(dt), r(*shape).to(dt))]

    def step(x, g, h0, z, dy, keep):
        out, h = F.glr_forward("mix", x, g, h0, out=keep[0], h_final=keep[1])
        F.groupnorm_forward(out, w, b, z, act="silu", y=keep[2])
        F.groupnorm_backward(out, dy, w, b, z, act="silu", dx=keep[3], dz=keep[4], dweight=keep[5], dbias=keep[6],
                             workspace=keep[7])
        F.glr_backward("mix", x, g, out, keep[3], h0, dx=keep[8], dg=keep[9], dh0=keep[10])

    def buffers():
        n = F.falcon_gn_bwd_workspace_bytes(F.make_seq_dims(*shape))
        e = lambda: torch.empty(shape, dtype=dt, device="cuda")  # noqa: E731
        f = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        return [e(), f(2, 3, 64), e(), e(), e(), f(3, 64), f(3, 64), torch.empty(n, dtype=torch.uint8, device="cuda"),
                e(), e(), f(2, 3, 64)]

    first, second = inputs(72), inputs(73)
    want = []
    for v in (first, second):
        keep = buffers()
        step(*v, keep)
        want.append(keep)
    torch.cuda.synchronize()

    static, keep = [t.clone() for t in first], buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(*static, keep)
    for v, ref in ((second, want[1]), (first, want[0]), (second, want[1])):
        for s, t in zip(static, v):
            s.copy_(t)
        for k in keep:
            k.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, r) in enumerate(zip(keep, ref)):
            assert i == 7 or torch.equal(a, r), i

    streams, kept = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(), buffers()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for s, v, k in zip(streams, (first, second), kept):
            with torch.cuda.stream(s):
                step(*v, k)
    torch.cuda.synchronize()
    for k, ref in zip(kept, want):
        for i, (a, r) in enumerate(zip(k, ref)):
            assert i == 7 or torch.equal(a, r), i


def test_falcon_read_through_the_norm_and_back():
    """A mixer as it is used: Falcon-1A's reads, normalised and gated into the projection's layout, and the whole
    backward pass; against the oracle's forward, 64-bit norm and the oracle's backward."""
    from oracle import falcon_bwd as OB
    from oracle import falcon_ref_fwd
    from weight_linear_attention_gb300 import inputs as I

    w = I.WORKLOADS[I.HEADLINE].with_(variant="falcon1a", dtype="f32", heads=2)
    T = 2 * w.chunk + 5
    inp = I.make_inputs(w, seed=5, seqlen=T, batch=2)
    d = {n: inp[n].cuda() for n in ("q", "k", "v", "beta", "lam")}
    r = Draw(80)
    z, dy = r(2, 2, T, 64), r(2, 2, T, 64)
    gw, gb = 1 + 0.1 * r(2, 64), 0.1 * r(2, 64)
    out, _, _ = F.forward(w.variant_id, d["q"], d["k"], d["v"], d["beta"], d["lam"], chunk=64)
    y = F.groupnorm_forward(out, gw.cuda(), gb.cuda(), z.cuda(), act="silu")
    assert y.transpose(1, 2).reshape(2, T, 128).data_ptr() == y.data_ptr()
    got = F.groupnorm_backward(out, dy.cuda(), gw.cuda(), gb.cuda(), z.cuda(), act="silu")
    grads = F.backward(w.variant_id, d["q"], d["k"], d["v"], d["beta"], d["lam"], got["dx"])

    # the norm against 64 bits of the same reads
    o = out.cpu()
    _close("y", y, *R.gn_forward(o, gw, gb, z, "silu"))
    ref, e = R.gn_backward(o, dy, gw, gb, z, "silu")
    for k in ref:
        _close(k, got[k], ref[k], e[k])
    # the chain against the oracles: the fp32 backward's own bound of 2e-4, plus what the reads' 1e-4 of
    # their largest moves the norm's gradient by
    ro, _, _ = falcon_ref_fwd(w.variant_id, inp["q"], inp["k"], inp["v"], inp["beta"], inp["lam"])
    assert abs(out.cpu().double().numpy() - ro).max() <= 1e-4 * abs(ro).max()
    want = OB.falcon_ref_bwd(w.variant_id, inp["q"], inp["k"], inp["v"], inp["beta"], inp["lam"],
                             got["dx"].cpu(), None, None)
    for k in ("dq", "dk", "dv", "dbeta", "dlam"):
        a = grads[k].cpu().double().numpy()
        assert abs(a - want[k]).max() <= 2e-4 * abs(want[k]).max(), k


def test_out_beside_its_inputs_in_one_buffer():
    """x, g and out as column blocks of one buffer, and one tensor as both inputs."""
    shape = (2, 3, 700, 64)
    x, g, h0 = glr_inputs("mix", shape, torch.bfloat16, 90)
    xd, gd, od = place("blocks", x, g, torch.full(shape, math.nan).to(torch.bfloat16))
    out, h = F.glr_forward("mix", xd, gd, h0.cuda(), out=od)
    (ro, rh), (eo, eh) = R.glr_forward("mix", x, g, h0)
    _close("out", out, ro, eo)
    _close("h_final", h, rh, eh)
    assert torch.equal(xd.cpu(), x) and torch.equal(gd.cpu(), g)  # the neighbours are as they were
    out, _ = F.glr_forward("mix", gd, gd, h0.cuda())
    _close("out", out, *[v[0] for v in R.glr_forward("mix", g, g, h0)])
    y = F.groupnorm_forward(xd, None, None, gd, act="silu", y=od)
    _close("y", y, *R.gn_forward(x, None, None, g, "silu"))
    assert torch.equal(xd.cpu(), x) and torch.equal(gd.cpu(), g)


def test_writes_stay_inside():
    """Outputs inside a larger buffer: every byte around them is as it was (cut channel tiles and last tiles)."""
    for shape in ((2, 1, 131, 40), (1, 2, 1, 72), (3, 1, 1300, 8)):
        B, H, T, d = shape
        x, g, h0 = glr_inputs("sigmoid", shape, torch.bfloat16, 91)
        w = Draw(92)(H, d).cuda()
        buf = torch.full((B, T + 3, H, d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
        view = buf[:, 1:T + 1, :, 8:8 + d].transpose(1, 2)
        xd, gd = x.cuda(), g.cuda()
        n = torch.tensor([T, 0, T // 2][:B], dtype=torch.int32, device="cuda")
        for write in (lambda: F.glr_forward("sigmoid", xd, gd, h0.cuda(), lengths=n, out=view),
                      lambda: F.groupnorm_forward(xd, w, None, gd, act="gelu", lengths=n, y=view),
                      lambda: F.glr_backward("sigmoid", xd, gd, xd, gd, lengths=n, dx=view),
                      lambda: F.groupnorm_backward(xd, gd, w, None, gd, act="gelu", lengths=n, dz=view)):
            buf.fill_(7.0)
            write()
            view.fill_(7.0)
            assert bool((buf == 7.0).all()), shape


def test_states_and_parameters_at_single_element_alignment():
    shape = (2, 3, 260, 64)
    x, g, h0 = glr_inputs("mix", shape, torch.bfloat16, 93)

    def off(t):
        return torch.empty(t.numel() + 1, device="cuda")[1:].view(t.shape).copy_(t)

    for T in (1, 260):
        xs, gs = x[:, :, :T].contiguous(), g[:, :, :T].contiguous()
        s = off(h0)
        out, h = F.glr_forward("mix", xs.cuda(), gs.cuda(), s, h_final=s)
        (ro, rh), (eo, eh) = R.glr_forward("mix", xs, gs, h0)
        _close("out", out, ro, eo)
        _close("h_final", h, rh, eh)
        got = F.glr_backward("mix", xs.cuda(), gs.cuda(), out, gs.cuda(), off(h0), dh0=off(h0))
        ref, e = R.glr_backward("mix", xs, gs, out.cpu(), gs, h0)
        for k, r, b in zip(("dx", "dg", "dh0"), ref, e):
            _close(k, got[k], r, b)
    w, b = Draw(94)(3, 64), Draw(95)(3, 64)
    _close("y", F.groupnorm_forward(x.cuda(), off(w), off(b)), *R.gn_forward(x, w, b))
    got = F.groupnorm_backward(x.cuda(), g.cuda(), off(w), off(b), dweight=off(w), dbias=off(b))
    ref, e = R.gn_backward(x, g, w, b)
    for k in ref:
        _close(k, got[k], ref[k], e[k])


def test_broadcast_norm_gate():
    """One gate row for all heads (stride 0): dz is that of every place."""
    shape = (2, 4, 33, 64)
    x, _, w, b, dy = gn_inputs(shape, torch.bfloat16, 96, False)
    z = Draw(97)(2, 1, 33, 64).to(torch.bfloat16)
    zd = z.cuda().expand(shape)
    y = F.groupnorm_forward(x.cuda(), w.cuda(), b.cuda(), zd, act="sigmoid")
    _close("y", y, *R.gn_forward(x, w, b, z.expand(shape), "sigmoid"))
    got = F.groupnorm_backward(x.cuda(), dy.cuda(), w.cuda(), b.cuda(), zd, act="sigmoid")
    ref, e = R.gn_backward(x, dy, w, b, z.expand(shape), "sigmoid")
    for k in ref:
        _close(k, got[k], ref[k], e[k])


@pytest.mark.parametrize("B,H,T", [(40, 6, 20), (300, 4, 50), (2, 2, 9), (64, 12, 16), (1, 1, 64)])
@pytest.mark.parametrize("gate", GATES)
def test_glr_short_sequences(gate, B, H, T):
    """Lengths around which the kernel changes, many sequences and few."""
    shape = (B, H, T, 64)
    x, g, h0 = glr_inputs(gate, shape, torch.bfloat16, 98)
    n = torch.tensor([(T * (i % 7)) // 6 for i in range(B)], dtype=torch.int32)
    out, h = run_fwd(gate, x, g, h0, n)
    (ro, rh), (eo, eh) = R.glr_forward(gate, x, g, h0, n)
    _close("out", out, ro, eo)
    _close("h_final", h, rh, eh)
    dout = Draw(99)(*shape).to(torch.bfloat16)
    dx, dg = poison("bthd", 2, shape, torch.bfloat16)
    got = F.glr_backward(gate, x.cuda(), g.cuda(), out, dout.cuda(), h0.cuda(), h0.cuda(), lengths=n.cuda(), dx=dx, dg=dg)
    ref, e = R.glr_backward(gate, x, g, out.cpu(), dout, h0, h0, n)
    for k, r, b in zip(("dx", "dg", "dh0"), ref, e):
        _close(k, got[k], r, b)


def test_first_call_of_a_process_inside_a_capture():
    """Nothing that a first call sets up breaks a capture."""
    import subprocess
    import sys

    code = """
import torch
from weight_linear_attention_gb300 import falcon as F
x = torch.randn(2, 3, 1500, 64, device="cuda").bfloat16()
z, h0 = torch.randn_like(x), torch.zeros(2, 3, 64, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, h = F.glr_forward("sigmoid", x, z, h0)
    y = F.groupnorm_forward(out, None, None, z, act="silu")
    d = F.groupnorm_backward(out, z, None, None, z, act="silu")
    e = F.glr_backward("sigmoid", x, z, out, d["dx"], h0)
graph.replay()
torch.cuda.synchronize()
want, _ = F.glr_forward("sigmoid", x, z, h0)
assert torch.equal(out, want) and torch.equal(y, F.groupnorm_forward(out, None, None, z, act="silu"))
assert torch.equal(e["dg"], F.glr_backward("sigmoid", x, z, out, d["dx"], h0)["dg"])
assert F.falcon_device_status() == F.FALCON_OK
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=240)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_host_threads():
    """Calls of two threads on streams of their own give what one thread's do."""
    import threading

    shape = (2, 3, 1200, 64)
    ins = [glr_inputs("mix", shape, torch.bfloat16, 100 + i) for i in range(2)]
    dev = [[t.cuda() for t in v] for v in ins]
    want = [F.glr_forward("mix", *v)[0] for v in dev]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(20):
                    out, _ = F.glr_forward("mix", *dev[i])
                    F.groupnorm_forward(out, act="silu")
            s.synchronize()
            got[i] = out
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert F.falcon_device_status() == F.FALCON_OK


def test_wrappers_refuse():
    x = torch.zeros(2, 2, 3, 8, device="cuda")
    for bad in (x[:, :, :, ::2], x.double(), x.cpu(), x[:, :1], x.transpose(2, 3)):
        with pytest.raises(ValueError):
            F.glr_forward("mix", x, bad)
    with pytest.raises(ValueError, match="contiguous"):
        F.glr_forward("mix", x[..., ::2], x[..., ::2])
    with pytest.raises(ValueError, match="gate"):
        F.glr_forward("tanh", x, x)
    with pytest.raises(ValueError, match="act"):
        F.groupnorm_forward(x, act="relu")
    with pytest.raises(ValueError, match="h0"):
        F.glr_forward("mix", x, x, torch.zeros(2, 8, device="cuda"))
    with pytest.raises(ValueError, match="lengths"):
        F.glr_forward("mix", x, x, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="weight"):
        F.groupnorm_forward(x, torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(F.FalconError):
        F.glr_forward("mix", x, x, out=x)
    with pytest.raises(F.FalconError):
        F.groupnorm_forward(x, eps=0.0)
