"""spec_verify_attn_kv8 on non-finite block and soft-prompt rows that are
seen, and non-finite queries: NaN for bf16 rows, what the arithmetic gives for
fp32 rows."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import Attn
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def call(dtype):
    return Attn(5, B=2, Hq=4, Hkv=2, R=9, S=(150, 40), n_soft=3, dtype=dtype, mask="tree", pad=False)


def outputs(a):
    a.run()
    assert bn.spec_get_status() == 0
    return a.o.double().cpu().numpy(), a.lse.double().cpu().numpy()


# what each place's readers are: (request, KV head) -> rows
def readers(a, where):
    return a.vis[0, :, 2] if where == "block" else a.sees[0]


def put(a, where, kv, x):
    """Element 5 of request 0's block row 2, or of soft-prompt row 1 (which
    request 1 sees too), in KV head 1."""
    if where == "block":
        (a.d_kb if kv == "k" else a.d_vb)[0, 1, 2, 5] = x
    else:
        (a.d_sk if kv == "k" else a.d_sv)[1, 1, 5] = x


@pytest.mark.parametrize("x", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["block", "soft"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys(dtype, where, x):
    a = call(dtype)
    want_o, want_l = outputs(a)
    put(a, where, "k", x)
    o, l = outputs(a)
    see = readers(a, where)
    assert see.any() and not see.all()
    # (not affected: heads 0 and 1, whose KV head is 0, and rows that do not see it)
    for h in range(4):
        for r in range(9):
            if h < 2 or not see[r]:
                assert np.array_equal(o[0, r, h], want_o[0, r, h]) and l[0, h, r] == want_l[0, h, r]
                continue
            if dtype == "f32" and not np.isnan(x) and a.q[0, r, h, 5] * x < 0:
                assert np.isfinite(o[0, r, h]).all() and l[0, h, r] < want_l[0, h, r] + 1e-6    # a score of -inf
            else:
                assert np.isnan(o[0, r, h]).all() and np.isnan(l[0, h, r])


@pytest.mark.parametrize("x", [NAN, INF, -INF])
@pytest.mark.parametrize("where", ["block", "soft"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values(dtype, where, x):
    a = call(dtype)
    want_o, want_l = outputs(a)
    put(a, where, "v", x)
    o, l = outputs(a)
    see = readers(a, where)
    assert np.allclose(l, want_l, rtol=2.0 ** -20, atol=1e-6)           # the scores are the keys' alone
    hit = np.zeros((9, 4), dtype=bool)
    hit[see, 2:] = True
    assert np.array_equal(o[0][~hit], want_o[0][~hit])
    if dtype == "bf16":
        assert np.isnan(o[0][hit]).all()
    else:
        other = np.arange(128) != 5
        assert np.array_equal(o[0][hit][:, other], want_o[0][hit][:, other])
        assert np.array_equal(o[0][hit][:, 5], np.full(int(hit.sum()), x), equal_nan=True)


@pytest.mark.parametrize("x", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries(dtype, x):
    a = call(dtype)
    want_o, want_l = outputs(a)
    a.d_q[0, 4, 3, 7] = x
    o, l = outputs(a)
    assert np.isnan(o[0, 4, 3]).all() and np.isnan(l[0, 3, 4])
    o[0, 4, 3], l[0, 3, 4] = want_o[0, 4, 3], want_l[0, 3, 4]
    assert np.array_equal(o, want_o) and np.array_equal(l, want_l)
