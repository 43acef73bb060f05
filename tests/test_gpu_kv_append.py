"""kv_append against the oracle: the whole cache, byte for byte."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import dev
from kv8_helpers import page_layout, to_storage, torch_dt
from oracle import chunk, kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def make(rng, paged, P, H, ps, d, dtype):
    shape = (P, H, d // 64, ps, 64) if paged else (P, H, ps, d)
    k, v = (to_storage(rng.standard_normal(shape), dtype) for _ in range(2))
    return k, v, dev(k).to(torch_dt(dtype)), dev(v).to(torch_dt(dtype))


def desc(paged, kc, vc):
    if not paged:
        return bn.kv_desc_contiguous(kc, vc)
    return bn.kv_desc_paged(kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("d,H,ps,n,pad", [(64, 1, 16, 1, 0), (128, 8, 16, 300, 0), (64, 3, 48, 77, 64),
                                          (128, 32, 128, 41, 8), (128, 5, 17 * 16, 130, 1024), (64, 2, 16, 0, 0)])
def test_append(dtype, paged, d, H, ps, n, pad):
    rng = np.random.default_rng(n + d)
    P = n // ps + 5
    k0, v0, kc, vc = make(rng, paged, P, H, ps, d, dtype)
    rows = to_storage(rng.standard_normal((n, 2 * H * d + pad)), dtype)
    r = dev(rows).to(torch_dt(dtype))
    slots = rng.permutation(P * ps)[:n].astype(np.int64)
    slots[rng.random(n) < 0.1] = -1
    k, v = (r[:, x * H * d:(x + 1) * H * d].unflatten(1, (H, d)) for x in (0, 1))
    bn.kv_append(desc(paged, kc, vc), k, v, dev(slots))
    assert bn.spec_get_status() == 0
    wk, wv = chunk.append_rows(k0, v0, rows[:, :H * d].reshape(n, H, d),
                               rows[:, H * d:2 * H * d].reshape(n, H, d), slots, paged)
    assert np.array_equal(kc.float().cpu().numpy(), wk) and np.array_equal(vc.float().cpu().numpy(), wv)


def test_slots_from_a_plan():
    rng = np.random.default_rng(5)
    H, d, ps, new, held = 2, 64, 16, np.array([40, 0, 1, 70], np.int32), np.array([5, 3, 16, 0], np.int32)
    n_pages, table, free = page_layout(rng, held, 8, ps, 12)
    k0, v0, kc, vc = make(rng, True, n_pages, H, ps, d, "bf16")
    tab, fh, cu = dev(table), dev(np.zeros(1, np.int32)), dev(np.zeros(5, np.int32))
    n = int(new.sum())
    slots = torch.empty(n, dtype=torch.int64, device="cuda")
    bn.spec_page_plan(ps, n_pages, dev(held), dev(new), tab, dev(free), fh, cu, slots)
    x = to_storage(rng.standard_normal((2, n, H, d)), "bf16")
    t = dev(x).to(torch.bfloat16)
    bn.kv_append(bn.kv_desc_paged(kc, vc, tab), t[0], t[1], slots)
    assert bn.spec_get_status() == 0
    want = kv8.page_plan(held, new, table, free, 0, ps, n)[3]
    wk, wv = chunk.append_rows(k0, v0, x[0], x[1], want, True)
    assert np.array_equal(kc.float().cpu().numpy(), wk) and np.array_equal(vc.float().cpu().numpy(), wv)


@pytest.mark.parametrize("paged", [True, False])
def test_slots_past_the_cache_are_skipped(paged):
    rng = np.random.default_rng(6)
    k0, v0, kc, vc = make(rng, paged, 3, 2, 16, 64, "f32")
    x = rng.standard_normal((2, 5, 2, 64)).astype(np.float32)
    slots = np.array([0, 48, 1 << 40, -(1 << 62), 47], dtype=np.int64)
    bn.kv_append(desc(paged, kc, vc), dev(x[0]), dev(x[1]), dev(slots))
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_PAGE
    ok = np.where((slots >= 0) & (slots < 48), slots, -1)
    wk, wv = chunk.append_rows(k0, v0, x[0], x[1], ok, paged)
    assert np.array_equal(kc.cpu().numpy(), wk) and np.array_equal(vc.cpu().numpy(), wv)


def test_bits_of_any_value_pass():
    """A copy: NaN payloads, infinities and subnormals arrive as they are."""
    bits = torch.randint(-2 ** 31, 2 ** 31 - 1, (2, 9, 2, 64), dtype=torch.int32, device="cuda")
    x = bits.view(torch.float32)
    kc, vc = torch.zeros((1, 2, 16, 64), device="cuda"), torch.zeros((1, 2, 16, 64), device="cuda")
    bn.kv_append(desc(False, kc, vc), x[0], x[1], torch.arange(9, device="cuda") + 4)
    assert torch.equal(kc.view(torch.int32)[0, :, 4:13].transpose(0, 1), bits[0])
    assert torch.equal(vc.view(torch.int32)[0, :, 4:13].transpose(0, 1), bits[1])
