"""The head norm's normal distribution function, from the constants as its source has them, against erfc in double."""

import os
import re

import torch

from weight_linear_attention_gb300 import build

SOURCE = os.path.join(build.CSRC, "falcon_gn.cuh")


def _constants():
    """kT and the polynomial's coefficients, rounded to fp32 as the compiler rounds them."""
    src = open(SOURCE).read()
    a, b = re.search(r"kT = ([\d.]+)f \* ([\d.]+)f", src).groups()
    c = re.search(r"constexpr float c\[10\] = \{([^}]*)\}", src).group(1)
    f = lambda v: torch.tensor(float(v), dtype=torch.float32)  # noqa: E731
    return (f(a) * f(b)).double(), torch.stack([f(v.strip().rstrip("f")) for v in c.split(",")]).double()


def test_normal_distribution_polynomial():
    """With t = 1 / (1 + kT v), t P(t) is exp(v^2 / 2) erfc(v / sqrt 2) to the relative errors that the source states."""
    k, c = _constants()
    assert len(c) == 10
    for top, most in ((5.0, 1.2e-7), (14.0, 1.4e-7), (1e6, 1.5e-7)):
        v = torch.linspace(0, top, 400001, dtype=torch.double)
        t = 1 / (1 + k * v)
        p = torch.zeros_like(t)
        for a in reversed(c):
            p = p * t + a
        error = float((t * p / torch.special.erfcx(v / 2 ** 0.5) - 1).abs().max())
        assert most / 1.2 < error <= most, (top, error)
