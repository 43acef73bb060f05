"""spec_rope refuses outputs that meet the positions or lengths it reads, without a
GPU (the pointers are never dereferenced on the host)."""

import pytest

from self_speculative_verification_gb300 import binding as bn
from test_chunk_host import INVALID, O, P, rope

LAUNCH = 5                # passed all checks: the launch alone fails without a GPU
FAR = 0x70000000


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("what is not refused would launch")
    return bn.load_library()


# q rows of 256 and k rows of 128 elements, 1024 apart, 6 of them; 24 bytes of
# positions, 8 of two lengths, 12 of their sums
@pytest.mark.parametrize("dt,es", [(bn.SPEC_BF16, 2), (bn.SPEC_F32, 4)])
@pytest.mark.parametrize("rows,width", [(O, 256), (O + 0x10000, 128)])
@pytest.mark.parametrize("what,length", [("pos", 24), ("seq", 8), ("cu", 12)])
def test_outputs_apart_from_what_says_where(lib, dt, es, rows, width, what, length):
    s, w = 1024 * es, width * es

    def call(at):
        kw = dict(pos=None, B=2, seq=FAR, cu=FAR + 0x1000) if what != "pos" else {}
        return rope(lib, dt=dt, **dict(kw, **{what: at}))

    for row in (0, 3, 5):
        first, last = rows + row * s, rows + row * s + w
        for at in (first - length + 4, first, first + 4, last - 4):
            assert call(at) == INVALID, (row, at - rows)
        # before it, and between it and the next
        assert call(first - length) == LAUNCH and call(last) == LAUNCH
    assert call(rows + 6 * s) == LAUNCH


@pytest.mark.parametrize("dt", [bn.SPEC_BF16, bn.SPEC_F32])
def test_what_is_not_read_may_lie_anywhere(lib, dt):
    assert rope(lib, dt=dt, pos=FAR, B=2, seq=O, cu=O) == LAUNCH          # positions are given
    assert rope(lib, dt=dt, Hk=0, sk=0, sko=0, pos=O + 0x10000) == LAUNCH  # there are no keys
