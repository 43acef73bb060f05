"""spec_rope at the ends of its row strides' range, without a GPU."""

import os
import subprocess
import sys

import pytest

from self_speculative_verification_gb300 import binding as bn
from test_chunk_host import INVALID, O, P, rope

LAUNCH = 5                # passed all checks: the launch alone fails without a GPU


@pytest.fixture(scope="module")
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("what is not refused would launch")
    return bn.load_library()


@pytest.mark.parametrize("dt", [bn.SPEC_BF16, bn.SPEC_F32])
@pytest.mark.parametrize("s", [1 << 62, 1 << 61, (1 << 63) - 8, 1 << 60])
def test_strides_past_the_address_space(lib, dt, s):
    """Their bytes do not fit 64 bits: refused, in place or not."""
    for kw in (dict(sq=s), dict(sqo=s), dict(sk=s), dict(sko=s), dict(sq=s, sqo=s, qo=P + 16),
               dict(sq=s, sqo=s, sk=s, sko=s), dict(sq=s, sqo=s, qo=P)):
        assert rope(lib, dt=dt, **kw) == INVALID, kw


@pytest.mark.parametrize("dt", [bn.SPEC_BF16, bn.SPEC_F32])
def test_the_stride_of_one_row_is_not_used(lib, dt):
    s = 1 << 62
    for kw in (dict(sq=s, sqo=s, sk=s, sko=s), dict(qo=P, sq=1024, sqo=s)):
        assert rope(lib, n=1, dt=dt, **kw) == LAUNCH, kw
    assert rope(lib, n=1, dt=dt, sq=s, sqo=s, qo=P + 16) == INVALID


def test_no_signal_ends_the_process():
    code = ("from test_chunk_host import P, rope\n"
            "from self_speculative_verification_gb300 import binding as bn\n"
            "lib = bn.load_library()\n"
            "for dt in (bn.SPEC_F32, bn.SPEC_BF16):\n"
            "    for s in (1 << 62, 1 << 61):\n"
            "        for qo in (P, P + 16):\n"
            "            assert rope(lib, dt=dt, sq=s, sqo=s, qo=qo) == 1\n")
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]), CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
