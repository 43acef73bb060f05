"""spec_verify_attn_kv8's bounded waits for every number of rows a unit can
have: the limit runs out, is reported, and the next call is right."""

import numpy as np
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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("R", [2, 4, 8, 16, 40])           # 8, 16, 32 and 64 rows; several blocks of 64
@pytest.mark.parametrize("long", [True, False])
def test_waits_run_out_and_the_next_call_is_right(long, R, d):
    if long:        # more tiles a CTA than ring slots
        a = Attn(R, B=4, Hq=32, Hkv=8, R=R, S=(9000, 8000, 8500, 7000), d=d, mask="chain", pad=False)
    else:           # many units a CTA
        a = Attn(R, B=60, Hq=32, Hkv=8, R=R, S=np.arange(60) * 9 % 300, d=d, mask="chain", pad=False)
    bn.spec_set_wait_limit(0)
    try:
        a.run()
        torch.cuda.synchronize()
    finally:
        bn.spec_set_wait_limit(-1)
    status = bn.spec_get_status()
    assert status & bn.SPEC_DEV_TIMEOUT, f"status {status:#x}"
    a.run()
    assert bn.spec_get_status() == 0
    a.check(requests=[0, 3], heads=[0, 31])
