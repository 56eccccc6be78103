"""Where the gated delta rule and the root-mean-square norm can go wrong beside their parity: what a call's parts leave for one
another, values that are not finite, operands' bits, decays of every strength."""

import pytest
import torch

from tests.test_gpu_block import DT, forward, inputs

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
