"""The 64-bit references of the strided operators against what defines them: autograd through a token loop,
central differences, and hand-worked values."""

import math

import pytest
import torch

from oracle import seq_ref as R


def _rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.double)


def test_glr_hand_worked():
    g = torch.log(torch.tensor([0.5, 0.25, 0.0])).view(1, 1, 3, 1)
    x = torch.tensor([1.0, 2.0, 3.0]).view(1, 1, 3, 1)
    (out, h), _ = R.glr_forward("decay", x, g, torch.tensor([[[4.0]]]))
    # 0.5*4+1, 0.25*3+2, a gate of -inf forgets
    assert torch.allclose(out.flatten(), torch.tensor([3.0, 2.75, 3.0], dtype=torch.double), atol=1e-7)
    assert torch.allclose(h.flatten(), out[0, 0, -1])
    (out, h), _ = R.glr_forward("mix", x, torch.zeros(1, 1, 3, 1), lengths=torch.tensor([2]))
    assert out.flatten().tolist() == [0.5, 1.25, 0.0] and h.item() == 1.25


@pytest.mark.parametrize("gate", ["decay", "sigmoid", "mix"])
@pytest.mark.parametrize("ragged", [False, True])
def test_glr_backward_is_the_gradient(gate, ragged):
    B, H, T, d = 3, 2, 7, 3
    x, h0 = _rand(B, H, T, d).requires_grad_(), _rand(B, H, d, seed=1).requires_grad_()
    g0 = _rand(B, H, T, d, seed=2)
    g = (-g0.abs() if gate == "decay" else g0).requires_grad_()
    dout, dh = _rand(B, H, T, d, seed=3), _rand(B, H, d, seed=4)
    n = torch.tensor([7, 0, 3]) if ragged else torch.tensor([T] * B)

    def loss(x, g, h0):
        h, total = h0, 0.0
        a = torch.exp(g) if gate == "decay" else torch.sigmoid(g)
        u = (1 - a) * x if gate == "mix" else x
        for t in range(T):
            ok = (t < n)[:, None, None]
            h = torch.where(ok, a[:, :, t] * h + u[:, :, t], h)
            total = total + (torch.where(ok, h, 0.0) * dout[:, :, t]).sum()
        return total + (h * dh).sum()

    want = torch.autograd.grad(loss(x, g, h0), (x, g, h0))
    (out, _), _ = R.glr_forward(gate, x.detach(), g.detach(), h0.detach(), n)
    got, _ = R.glr_backward(gate, x.detach(), g.detach(), out, dout, h0.detach(), dh, n)
    for a, b in zip(got, want):
        assert torch.allclose(a, b, atol=1e-13)
    # central differences: third derivatives times step^2 / 6, and 1e-16 / step of rounding
    step = 1e-5
    for k, v in enumerate((x, g, h0)):
        way = _rand(*v.shape, seed=9 + k)
        args = [t.detach() for t in (x, g, h0)]
        hi, lo = list(args), list(args)
        hi[k], lo[k] = args[k] + step * way, args[k] - step * way
        slope = (loss(*hi) - loss(*lo)) / (2 * step)
        assert abs(slope - (got[k] * way).sum()) < 1e-7 * (1 + abs(slope))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("gated", [False, True])
def test_gn_backward_is_the_gradient(act, gated):
    B, H, T, d = 2, 3, 4, 5
    x, w, b = _rand(B, H, T, d).requires_grad_(), _rand(H, d, seed=1).requires_grad_(), _rand(H, d, seed=2).requires_grad_()
    z = _rand(B, H, T, d, seed=3).requires_grad_() if gated else None
    dy, n = _rand(B, H, T, d, seed=4), torch.tensor([4, 2])

    def loss(x, w, b, z):
        y, _ = R.gn_forward(x, w, b, z, act, 1e-5, n)
        return (y * dy).sum()

    leaves = [x, w, b] + ([z] if gated else [])
    want = torch.autograd.grad(loss(x, w, b, z), leaves)
    got, _ = R.gn_backward(x.detach(), dy, w.detach(), b.detach(), None if z is None else z.detach(), act, 1e-5, n)
    for name, v in zip(("dx", "dweight", "dbias", "dz"), want):
        assert torch.allclose(got[name], v, atol=1e-11), name
    step, way = 1e-5, _rand(B, H, T, d, seed=7)
    args = [v.detach() for v in (x, w, b)] + [None if z is None else z.detach()]
    slope = (loss(args[0] + step * way, *args[1:]) - loss(args[0] - step * way, *args[1:])) / (2 * step)
    assert abs(slope - (got["dx"] * way).sum()) < 1e-6 * (1 + abs(slope))


def test_gn_hand_worked():
    x = torch.tensor([1.0, 3.0]).view(1, 1, 1, 2)
    y, _ = R.gn_forward(x, torch.tensor([[2.0, 2.0]]), torch.tensor([[0.0, 1.0]]), eps=3.0)  # var 1, + eps 3: sd 2
    assert y.flatten().tolist() == [-1.0, 2.0]
    y, _ = R.gn_forward(x, z=torch.zeros(1, 1, 1, 2), name="sigmoid", eps=3.0)
    assert y.flatten().tolist() == [-0.25, 0.25]
    y, _ = R.gn_forward(x, z=torch.full((1, 1, 1, 2), math.nan), lengths=torch.tensor([0]))
    assert y.flatten().tolist() == [0.0, 0.0]


def test_close_counts_a_rounding():
    v = torch.tensor([1.0 + 2.0 ** -9], dtype=torch.double)
    assert R.close(v.to(torch.bfloat16), v, torch.zeros(1))[0]
    assert not R.close(v.to(torch.bfloat16) + 2.0 ** -6, v, torch.zeros(1))[0]
    nan = torch.tensor([math.nan], dtype=torch.double)
    assert R.close(nan.float(), nan, nan)[0] and not R.close(torch.zeros(1), nan, nan)[0]
    assert not R.close(nan.float(), torch.zeros(1, dtype=torch.double), torch.zeros(1))[0]
