"""kv8_append and kv8_commit on pages that held something before: recycled
ones, and ones whose scales the writers did not give."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import TABLE, pack, random_cache, to_storage, torch_dt, unpack
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("was", [float("nan"), 2.0 ** 40])
def test_a_recycled_page_is_begun_by_its_first_token(dtype, was):
    """Page 1's former owner left scales that are NaN or far too large.  A
    chunk that writes the token at offset 0 begins the page anew; one whose
    token there is not written goes on with what the page holds."""
    rng = np.random.default_rng(3)
    H, d, ps = 2, 128, 16
    codes, scales = random_cache(rng, 3, H, ps, d)
    scales[1] = was
    x = to_storage(rng.standard_normal((20, H, d)), dtype)
    for first in (10, -1):
        slots = np.arange(20, dtype=np.int64) + 10          # offset 10 of page 0 on
        if first < 0:
            slots[6] = -1                                   # offset 0 of page 1
        kv, sc = pack(codes), dev(scales)
        bn.kv8_append(bn.kv8_desc(kv, sc), dev(x).to(torch_dt(dtype)), dev(x).to(torch_dt(dtype)), dev(slots))
        assert bn.spec_get_status() == 0
        c, s = kv8.append(TABLE[codes], scales.astype(np.float64), x, x, slots, ps)
        got, gs = TABLE[unpack(kv)], sc.double().cpu().numpy()
        assert np.array_equal(got, c) and np.array_equal(gs, s, equal_nan=True)
        if first < 0:
            assert np.array_equal(gs[1], scales[1], equal_nan=True)
        else:                                               # within half a step of the new rows
            assert np.all(gs[1] <= 2.0 ** -6)
            assert np.all(np.abs(got[1, :, 0, :14] * gs[1, :, 0, None, None] - x[6:].transpose(1, 0, 2))
                          <= 2.0 ** -4 * np.abs(x[6:].transpose(1, 0, 2)) + gs[1].max() * 2.0 ** -10)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("writer", ["append", "commit"])
def test_scales_outside_the_readers_range(writer, d, dtype):
    """Scales that the writers did not give count for them as for the reader:
    below 2^-60 (0 and negative ones too) as 2^-60, above 2^60 as 2^60."""
    rng = np.random.default_rng(4)
    H, ps, n = 3, 32, 5
    odd = np.array([0.0, -1.0, 2.0 ** -70, 2.0 ** 70, 2.0 ** -100, 3e38], dtype=np.float32)
    codes, scales = random_cache(rng, len(odd), H, ps, d)
    scales[:] = odd[:, None, None]
    size = np.float32(2.0) ** rng.choice([-64, -60, -55, -3, 4, 50], size=(len(odd) * n, H, 1))
    x = to_storage(rng.standard_normal((len(odd) * n, H, d)) * size, dtype)
    at = np.concatenate([p * ps + 9 + np.arange(n) for p in range(len(odd))]).astype(np.int64)
    kv, sc, dx = pack(codes), dev(scales), dev(x).to(torch_dt(dtype))
    as_read = np.clip(scales.astype(np.float64), 2.0 ** -60, 2.0 ** 60)
    if writer == "append":
        bn.kv8_append(bn.kv8_desc(kv, sc), dx, dx, dev(at))
    else:                                                   # every page a request with nine tokens
        table = dev(np.arange(len(odd), dtype=np.int32)[:, None])
        kb = dx.view(len(odd), n, H, d).transpose(1, 2).contiguous()
        i32 = dict(dtype=torch.int32, device="cuda")
        path = torch.arange(n, **i32).repeat(len(odd), 1)
        seq = torch.full((len(odd),), 9, **i32)
        bn.kv8_commit(bn.kv8_desc(kv, sc, table), kb, kb, path, torch.full_like(seq, n), seq,
                      torch.zeros(1, **i32), torch.zeros(1, **i32))
        assert seq.tolist() == [9 + n] * len(odd)
    assert bn.spec_get_status() == 0
    c, s = kv8.append(TABLE[codes], as_read, x, x, at, ps)
    assert np.array_equal(TABLE[unpack(kv)], c) and np.array_equal(sc.double().cpu().numpy(), s)
