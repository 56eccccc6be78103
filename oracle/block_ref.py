"""64-bit references of the gated delta rule and the root-mean-square norm, token by token from their definitions.

Inputs are CPU tensors of any type; everything is computed in double from their values."""

import math

import torch

U = 2.0 ** -24

# What fp32 arithmetic may make of a delta rule result at worst, relative to the largest norm of what is summed for it. A
# product over 64 or 128 terms is at most 48 sums on the tensor cores (16 steps of 8 in three passes), each of which may drop
# a unit (2 U); at most eight products follow one another from the inputs to a gradient (the Gram matrix, the inverse's
# two levels of two, E, a score, the result), and the errors of at most three of the operands of one meet: 48 x 2 x 8 x 3 U.
GDR = 2304 * U
# From bf16 inputs, too: all operands have fp32's 24 bits.
GDR_BF16 = GDR_BF16_DK = GDR

# What it makes of a whole head's tensor, in the 2-norm, where no error is at its worst and few have one sign: a product leaves
# about 4 U (its operands' 24 bits and the planes' products that are left out, 2^-24 each, and sums that are cut four times),
# eight in a row sqrt(8) times that, 11 U. Three times that is the bound; operands of 16 bits leave 2^-17 = 128 U and more.
NEAR = 32 * U
# dg adds up to 64 terms of its chunk, 32 in the middle, whose errors add as their root: six times a term's, of which
# each has that of one product of fp32 results, 8 U; half as much again.
NEAR_DG = 72 * U


def _live(lengths, B, T):
    n = torch.full((B,), T) if lengths is None else lengths.long().clamp(0, T)
    return torch.arange(T)[:, None] < n[None, :]  # [T,B]


def _shared(t, H):
    return t.double().repeat_interleave(H // t.shape[1], 1) if t.shape[1] != H else t.double()


def gdr_forward(q, k, v, beta, g, S0=None, *, scale=None, lengths=None, keep=False):
    """(out, S_final), or with `keep` also the state before each token."""
    B, H, T, dv = v.shape
    dk = q.shape[-1]
    scale = dk ** -0.5 if scale is None else scale
    live = _live(lengths, B, T)
    q, k, v, beta, a = _shared(q, H), _shared(k, H), v.double(), beta.double(), torch.exp(g.double())
    S = torch.zeros(B, H, dk, dv, dtype=torch.double) if S0 is None else S0.double()
    out, before = torch.zeros(B, H, T, dv, dtype=torch.double), []
    for t in range(T):
        before.append(S)
        kept = a[:, :, t, None, None] * S
        err = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", kept, k[:, :, t])
        new = kept + k[:, :, t, :, None] * (beta[:, :, t, None] * err)[:, :, None]
        o = scale * torch.einsum("bhkv,bhk->bhv", new, q[:, :, t])
        on = live[t][:, None, None]
        out[:, :, t] = torch.where(on, o, 0.0)
        S = torch.where(on[..., None], new, S)
    return (out, S, before) if keep else (out, S)


def gdr_backward(q, k, v, beta, g, dout, S0=None, dS_final=None, *, scale=None, lengths=None):
    """dict dq, dk, dv, dbeta, dg, dS0."""
    B, H, T, dv_ = v.shape
    Hk, dk_ = q.shape[1], q.shape[-1]
    scale = dk_ ** -0.5 if scale is None else scale
    live = _live(lengths, B, T)
    _, S, before = gdr_forward(q, k, v, beta, g, S0, scale=scale, lengths=lengths, keep=True)
    q, k, v, beta, a, dout = _shared(q, H), _shared(k, H), v.double(), beta.double(), torch.exp(g.double()), dout.double()
    D = torch.zeros_like(S) if dS_final is None else dS_final.double()
    r = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v), "dbeta": torch.zeros_like(beta),
         "dg": torch.zeros_like(beta)}
    for t in reversed(range(T)):
        kt, bt, at = k[:, :, t], beta[:, :, t, None], a[:, :, t, None, None]
        kept = at * before[t]
        err = v[:, :, t] - torch.einsum("bhkv,bhk->bhv", kept, kt)
        new = kept + kt[..., None] * (bt * err)[:, :, None]
        total = D + scale * q[:, :, t, :, None] * dout[:, :, t, None]
        pulled = torch.einsum("bhkv,bhk->bhv", total, kt)
        derr = bt * pulled
        dkept = total - kt[..., None] * derr[:, :, None]
        on = live[t][:, None]

        def note(name, x):
            r[name][:, :, t] = torch.where(on if x.dim() == 2 else on[..., None], x, 0.0)

        note("dq", scale * torch.einsum("bhkv,bhv->bhk", new, dout[:, :, t]))
        note("dk", torch.einsum("bhkv,bhv->bhk", total, bt * err) - torch.einsum("bhkv,bhv->bhk", kept, derr))
        note("dv", derr)
        note("dbeta", (pulled * err).sum(-1))
        note("dg", (dkept * kept).sum((-1, -2)))
        D = torch.where(on[..., None, None], at * dkept, D)
    for name in ("dq", "dk"):
        if Hk != H:
            r[name] = r[name].view(B, Hk, H // Hk, T, dk_).sum(2)
    return dict(r, dS0=D)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def gdr_close(got, want, room, dtype=torch.float32):
    """Whether `got` is within its type's rounding and `room` of the rows' largest norm, in the 2-norm of every row
    (the last axis; a [B,H,T] tensor is one row a head). Returns it and the share of the bound that was used."""
    got, want = got.detach().cpu().double(), want.double()
    if got.shape != want.shape:
        return False, math.inf
    if not want.numel():
        return True, 0.0
    if not torch.equal(torch.isfinite(got), torch.isfinite(want)):
        return False, math.inf
    norm = want.norm(dim=-1)
    top = norm.amax(-1, keepdim=True)
    bound = half_step(dtype) * norm + room * top + 1e-30
    share = ((got - want).norm(dim=-1) / bound).max().item()
    return share <= 1, share


def gdr_near(got, want, dtype=torch.float32, room=NEAR, size=None):
    """The share that the error of a [B,H,...] tensor has of `room`, head by head in the 2-norm; `size` [B,H]: the norm of
    what was summed for it, where that is more than the result.

    Of what is rounded to bf16 only that shows which goes past half a step of the rounding: value by value that is at most
    the error before it, five standard deviations of 11 U of its row (of its head, where that has more): 2 room."""
    got, want = got.detach().cpu().double(), want.double()
    norm = want.flatten(2).norm(dim=-1) if size is None else size
    if dtype == torch.float32:
        return ((got - want).flatten(2).norm(dim=-1) / (room * norm + 1e-300)).max().item()
    top = torch.maximum(got.abs(), want.abs()).clamp(min=2.0 ** -126)
    past = (got - want).abs() - torch.exp2(torch.floor(torch.log2(top))) * half_step(dtype)
    d = want.shape[-1]
    rms = torch.maximum(want.norm(dim=-1) / d ** 0.5, norm[..., None] / (want[0, 0].numel()) ** 0.5)[..., None]
    return (past / (2 * room * rms + 1e-300)).max().item()


def cut(x, bits):
    """x in fp32 with that many leading bits of its mantissa (the first of them implied), the others cut off."""
    return (x.float().contiguous().view(torch.int32) & -(1 << (24 - bits))).view(torch.float32)


def rms_forward(x, weight=None, residual=None, *, eps=1e-6, lengths=None):
    """(y, h) of [B,T,d], y in double."""
    B, T, d = x.shape
    live = _live(lengths, B, T).T[..., None]
    h = x if residual is None else (x.double() + residual.double()).to(x.dtype)
    hd = torch.where(live, h.double(), 0.0)
    y = hd / torch.sqrt(hd.square().mean(-1, keepdim=True) + eps) * (1.0 if weight is None else weight.double())
    return torch.where(live, y, 0.0), torch.where(live, h, torch.zeros_like(h))


def rms_room(d):
    """Relative error of y in fp32: a sum of squares adds a lane's 32 and then 5 or 9 levels (and up to 16 warps), its
    root halves that; the root, quotient, mean and two products add 6 roundings."""
    return (0.5 * (32 + 9 + 16 + 2) + 6) * U


def rms_backward(h, dy, weight=None, dh=None, *, eps=1e-6, lengths=None):
    """((dx, dweight), and their rounding errors' bounds)."""
    B, T, d = h.shape
    live = _live(lengths, B, T).T[..., None]
    h, dy = torch.where(live, h.double(), 0.0), torch.where(live, dy.double(), 0.0)
    w = torch.ones(d, dtype=torch.double) if weight is None else weight.double()
    rstd = 1 / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    p = dy * w
    own = rstd * p
    pull = rstd ** 3 * h * (p * h).mean(-1, keepdim=True)
    dx = own - pull
    e = 2 * rms_room(d)
    # the mean of p h is off by that much of the mean of |p h|
    bound = e * own.abs() + 3 * e * rstd ** 3 * h.abs() * (p * h).abs().mean(-1, keepdim=True)
    if dh is not None:
        dh = torch.where(live, dh.double(), 0.0)
        dx = dx + dh
        bound = bound + U * (dh.abs() + dx.abs())
    n = dy * h * rstd
    rows = B * T
    deep = rows // (4 * 304) + rows // 304 + 4 + 40 + 10  # a lane's, its CTA's and the last sum's additions
    return (dx, n.sum((0, 1))), (bound, (e + deep * U) * n.abs().sum((0, 1)))


def e4m3(x):
    """The nearest e4m3 value (ties to even) of each |x| <= 448, in double."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step
