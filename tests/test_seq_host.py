"""Host-only checks of the strided operators (falcon_glr_*, falcon_gn_*): every call below is refused by the
synchronous argument check, or has nothing to do, so nothing is launched."""

import math

import pytest
import torch

from weight_linear_attention_gb300 import build as fbuild
from weight_linear_attention_gb300 import falcon as F

A = 1 << 40  # fake device addresses: never dereferenced
GB = 1 << 30
INV, UNS, MIS = F.FALCON_ERR_INVALID_ARG, F.FALCON_ERR_UNSUPPORTED, F.FALCON_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def lib():
    fbuild.build()
    return F.load()


def _dims(b=2, h=3, t=5, d=64, dtype=F.FALCON_BF16):
    return F.make_seq_dims(b, h, t, d, dtype=dtype)


def glr(gate=0, dims=None, strides=None, x=A, g=A + GB, h0=None, lengths=None, out=A + 2 * GB, h_final=None):
    return F.falcon_glr_fwd(gate, x, g, h0, lengths, out, h_final, dims or _dims(), strides, stream=0)


def glr_b(gate=2, dims=None, strides=None, **kw):
    p = dict(x=A, g=A + GB, out=A + 2 * GB, h0=None, lengths=None, dout=A + 3 * GB, dh_final=None, dx=A + 4 * GB,
             dg=A + 5 * GB, dh0=None)
    p.update(kw)
    return F.falcon_glr_bwd(gate, p["x"], p["g"], p["out"], p["h0"], p["lengths"], p["dout"], p["dh_final"], p["dx"],
                            p["dg"], p["dh0"], dims or _dims(), strides, stream=0)


def gn(act=1, dims=None, strides=None, eps=1e-5, **kw):
    p = dict(x=A, z=A + GB, weight=None, bias=None, lengths=None, y=A + 2 * GB)
    p.update(kw)
    return F.falcon_gn_fwd(act, p["x"], p["z"], p["weight"], p["bias"], p["lengths"], p["y"], dims or _dims(), strides,
                           eps, stream=0)


def gn_b(act=1, dims=None, strides=None, eps=1e-5, ws=A + 9 * GB, ws_bytes=None, **kw):
    dims = dims or _dims()
    p = dict(x=A, z=A + GB, weight=None, bias=None, lengths=None, dy=A + 2 * GB, dx=A + 3 * GB, dz=A + 4 * GB,
             dweight=A + 5 * GB, dbias=A + 6 * GB)
    p.update(kw)
    if ws_bytes is None:
        ws_bytes = F.falcon_gn_bwd_workspace_bytes(dims)
    return F.falcon_gn_bwd(act, p["x"], p["z"], p["weight"], p["bias"], p["lengths"], p["dy"], p["dx"], p["dz"],
                           p["dweight"], p["dbias"], dims, strides, eps, ws, ws_bytes, stream=0)


CALLS = [glr, glr_b, gn, gn_b]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("dims,want", [
    (_dims(b=-1), INV), (_dims(h=-2), INV), (_dims(t=-1), INV), (_dims(d=0), INV), (_dims(d=-4), INV),
    (_dims(dtype=2), UNS), (_dims(t=1 << 30), UNS), (_dims(b=1 << 31), UNS), (_dims(h=1 << 31), UNS),
    (_dims(b=1 << 30, h=1 << 30, d=1 << 30), UNS),
])
def test_sizes(call, dims, want):
    assert call(dims=dims) == want


def test_reserved_field_and_missing_dims():
    d = _dims()
    d.reserved = 1
    assert glr(dims=d) == INV
    assert F.load().falcon_glr_fwd(0, A, A + GB, None, None, A + 2 * GB, None, None, None, 0) == INV
    assert F.load().falcon_gn_bwd_workspace_bytes(None) == 0


def test_choices():
    for gate in (-1, 3):
        assert glr(gate=gate) == INV and glr_b(gate=gate) == INV
    for act in (-1, 4):
        assert gn(act=act) == INV and gn_b(act=act) == INV
    for eps in (0.0, -1e-5, math.nan, math.inf):
        assert gn(eps=eps) == INV and gn_b(eps=eps) == INV
    assert gn(dims=_dims(d=1025)) == UNS and gn_b(dims=_dims(d=1025)) == UNS


def test_sizes_without_a_kernel():
    far = dict(x=A, g=A + (1 << 50), out=A + (2 << 50))
    assert glr(dims=_dims(b=1 << 30, h=4, t=16, d=64), **far) == UNS           # more channel tiles than a grid takes
    assert glr(dims=_dims(b=1 << 30, h=1 << 20, t=1, d=64), x=A, g=A + (1 << 60), out=A + (2 << 60)) == UNS
    assert gn(dims=_dims(b=1 << 20, h=1 << 10, t=1 << 10), z=None, y=A + (1 << 50)) == UNS  # 2^40 rows
    assert gn_b(dims=_dims(h=70000), z=None, dz=None, dy=A + (1 << 40), dx=A + (2 << 40), dweight=None,
                dbias=None) == UNS


def test_missing_tensors():
    for k in ("x", "g", "out"):
        assert glr(**{k: None}) == INV, k
    for k in ("x", "g", "out", "dout", "dx", "dg"):
        assert glr_b(**{k: None}) == INV, k
    for k in ("x", "y"):
        assert gn(**{k: None}) == INV, k
    for k in ("x", "dy", "dx"):
        assert gn_b(**{k: None}) == INV, k
    assert gn_b(dz=None) == INV and gn_b(z=None) == INV  # a gate and its gradient come together


def test_alignment():
    for k in ("x", "g", "out"):
        assert glr(**{k: A + 7 * GB + 1}) == MIS, k
    for k in ("h0", "lengths", "h_final"):
        assert glr(**{k: A + 7 * GB + 2}) == MIS, k
    assert glr(dims=_dims(dtype=F.FALCON_F32), x=A + 2) == MIS
    assert gn(weight=A + 7 * GB + 2) == MIS
    assert gn_b(ws=A + 9 * GB + 128) == MIS


def test_workspace():
    n = F.falcon_gn_bwd_workspace_bytes(_dims())
    assert n > 0 and n % (2 * 3 * 64 * 4) == 0
    assert gn_b(ws_bytes=n - 1) == INV and gn_b(ws=None) == INV
    for d in (_dims(t=0), _dims(b=0), _dims(h=0), _dims(d=2000), _dims(dtype=5)):
        assert F.falcon_gn_bwd_workspace_bytes(d) == 0
    assert gn_b(ws=A + 2 * GB) == INV  # on dy


def test_written_buffers_overlap_nothing():
    assert glr(out=A) == INV                                    # in place
    assert glr(out=A + 128) == INV
    assert glr(h_final=A + 2 * GB) == INV                       # on out
    assert glr(h0=A + 3 * GB, h_final=A + 3 * GB + 16) == INV   # only exactly in place
    assert glr(lengths=A + 2 * GB) == INV
    assert glr_b(dx=A + 5 * GB) == INV and glr_b(dg=A + 3 * GB) == INV
    assert glr_b(h0=A + 6 * GB, dh0=A + 6 * GB) == INV          # the backward has no in-place state
    assert gn(y=A + GB) == INV and gn_b(dz=A + 3 * GB) == INV
    assert gn_b(dweight=A + 6 * GB) == INV


def test_strides_that_are_refused():
    dense = [3 * 5 * 64, 5 * 64, 64]
    assert glr(strides=dense * 2 + [0, 5 * 64, 64]) == INV       # two sequences on one output
    assert glr(strides=dense * 2 + [3 * 5 * 64, 5 * 64, 63]) == INV
    assert glr(strides=dense * 2 + [960, 320, -64]) == INV
    assert glr(strides=[-960, 320, 64] + dense * 2) == INV
    assert glr(strides=dense * 2 + [1 << 62, 320, 64]) == INV    # leaves the address space
    assert glr(strides=dense * 2 + [320, 320, 64]) == INV        # heads and sequences on one another
    # column blocks of one buffer that reach into each other: blocks of 192 at an offset of 128 elements
    block = [5 * 384, 64, 384]
    assert glr(strides=block * 3, x=A, g=A + 384, out=A + 256, dims=_dims()) == INV
    # three blocks of 192 in rows of 384: the third starts where the next token's first does
    assert glr(strides=block * 3, x=A, g=A + 384, out=A + 768, dims=_dims()) == INV


@pytest.mark.parametrize("call", CALLS)
def test_nothing_to_do_launches_nothing(call):
    none = dict(dweight=None, dbias=None) if call is gn_b else {}  # given, they would be set to zero
    for d in (_dims(b=0), _dims(h=0)):
        assert call(dims=d, **none) == F.FALCON_OK
    assert glr(dims=_dims(b=0), x=None, g=None, out=None) == F.FALCON_OK
    assert gn(dims=_dims(t=0), x=None, z=None, y=None) == F.FALCON_OK


def test_wrappers_check_tensors():
    x = torch.zeros(1, 1, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        F.glr_forward("mix", x, x)
    with pytest.raises(ValueError, match="B,H,T,d"):
        F.groupnorm_forward(x[0])
