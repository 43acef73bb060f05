"""spec_rope at far positions with frequencies of either sign, pair by pair."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import dev
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def angle(f, pos):
    """f pos less whole turns, of the double f, in 60 digits."""
    a = Decimal(f) * pos
    turns = (a / (2 * PI)).to_integral_value()
    return float(a - 2 * PI * turns)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
@pytest.mark.parametrize("layout", [bn.SPEC_ROPE_PAIRS, bn.SPEC_ROPE_HALVES])
@pytest.mark.parametrize("what", ["whole turns", "slow"])
def test_small_frequencies_far_away(sign, layout, what):
    """x = 1, y = 0 becomes (cos t, sin t).  The angle is off by 2^-24 of a half turn
    and the frequency by 2^-52 of itself; sin and cos by two units of theirs (2^-22 of
    themselves) and a rounding each in the factor, the products and the sum (2^-24,
    counted as 2^-22 together)."""
    d, half = 256, 128
    pos = np.array([2 ** 31 - 1, 2 ** 31 - 12345, 1999999973, 5], dtype=np.int32)
    k = np.arange(1, half + 1)
    # that many whole turns over the first position, where sin t tells a small angle
    # exactly; or from 10^-14 on
    f = sign * (2 * np.pi * k / float(pos[0]) if what == "whole turns" else 10.0 ** (-14 + k / 16.0))
    x = np.zeros((len(pos), 1, d), dtype=np.float32)
    first = np.arange(0, d, 2) if layout == bn.SPEC_ROPE_PAIRS else np.arange(half)
    second = first + (1 if layout == bn.SPEC_ROPE_PAIRS else half)
    x[..., first] = 1.0
    q = dev(x)
    out = torch.empty_like(q)
    bn.spec_rope(bn.rope_desc(len(pos), 1, 0, d, d, layout, bn.SPEC_F32), f.tolist(), q, out, positions=dev(pos))
    got = out.double().cpu().numpy()[:, 0]
    t = np.array([[angle(float(fi), int(p)) for fi in f] for p in pos])
    off = np.pi * 2.0 ** -24 + 2.0 ** -52 * np.abs(f[None] * pos[:, None])
    for i, want, slope in ((second, np.sin(t), np.cos(t)), (first, np.cos(t), np.sin(t))):
        bound = off * np.abs(slope) + off ** 2 + 2.0 ** -21 * np.abs(want)
        e = np.abs(got[:, i] - want) / bound
        assert e.max() <= 1, f"off by {e.max()} of its bound"
