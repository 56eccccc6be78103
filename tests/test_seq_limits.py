"""The sizes at which the header says that the sequence operators refuse a call; refused on the host, before anything is
launched (the addresses are never used)."""

import pytest

from weight_linear_attention_gb300 import build as fbuild
from weight_linear_attention_gb300 import falcon as F

A = 1 << 40
FAR = 1 << 58  # between tensors: beyond any of the extents below
UNS = F.FALCON_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    fbuild.build()
    F.load()


def _glr(dims, strides=None):
    return F.falcon_glr_fwd(1, A, A + FAR, None, None, A + 2 * FAR, None, dims, strides, stream=0)


def _glr_bwd(dims):
    t = [A + i * FAR for i in range(6)]
    return F.falcon_glr_bwd(2, t[0], t[1], t[2], None, None, t[3], None, t[4], t[5], None, dims, stream=0)


@pytest.mark.parametrize("call", [_glr, _glr_bwd])
@pytest.mark.parametrize("b,h,t,d", [
    (1 << 15, 1 << 15, 9, 64),      # heads are T apart: B H items of one tile of channels
    (1 << 15, 1 << 14, 300, 65),    # two tiles each
    (1 << 20, 1, 300, 1 << 16),     # one head of many channels
    (1 << 22, 1 << 10, 8, 1 << 8),  # few tokens: by the channels in all
])
def test_recurrence(call, b, h, t, d):
    assert call(F.make_seq_dims(b, h, t, d)) == UNS


def test_recurrence_heads_side_by_side():
    """Heads without a gap are one head of H d channels, in as many tiles of 64."""
    b, h, t, d = 1 << 10, 1 << 20, 9, 64
    layout = [t * h * d, d, h * d]
    assert _glr(F.make_seq_dims(b, h, t, d), layout * 3) == UNS


def _gn(dims):
    return F.falcon_gn_fwd(0, A, None, None, None, None, A + FAR, dims, stream=0)


def _gn_bwd(dims):
    return F.falcon_gn_bwd(0, A, None, None, None, None, A + FAR, A + 2 * FAR, None, None, None, dims, stream=0)


def test_norm():
    assert _gn(F.make_seq_dims(1, 1 << 30, 1, 1)) == UNS
    assert _gn(F.make_seq_dims(1 << 10, 1 << 10, 1 << 11, 1)) == UNS   # 2^31 rows
    assert _gn_bwd(F.make_seq_dims(2, 1, (1 << 30) - (1 << 15), 1)) == UNS
    assert _gn_bwd(F.make_seq_dims(1, 1 << 16, 1, 1)) == UNS
