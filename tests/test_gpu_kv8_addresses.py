"""spec_verify_attn_kv8 with arrays at addresses of their type's own alignment."""

import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import Attn
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def one_on(t):
    """The same contiguous tensor, one element past an aligned address."""
    buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 5, 20])
def test_arrays_one_element_past_an_aligned_address(R, dtype):
    a = Attn(R, B=3, Hq=8, Hkv=2, R=R, S=(300, 17, 90), n_soft=3, mask="tree", dtype=dtype)
    a.run()
    want = a.o.clone(), a.lse.clone()
    for name in ("d_scales", "d_table", "d_S", "d_vis", "d_flags", "lse"):
        setattr(a, name, one_on(getattr(a, name)))
    assert a.d_scales.data_ptr() % 8 == 4
    a.cache = bn.kv8_desc(a.d_kv, a.d_scales, a.d_table)
    a.o.zero_()
    a.lse.zero_()
    a.run()
    assert bn.spec_get_status() == 0
    assert torch.equal(a.o, want[0]) and torch.equal(a.lse, want[1])
