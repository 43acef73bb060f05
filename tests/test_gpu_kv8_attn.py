"""spec_verify_attn_kv8 against the float64 oracle on the cache's values:
head layouts, lengths from nothing to many tiles, pages of every kind, masks
that leave a row empty, soft prompts, both types, odd scales; slots that no
token holds carry NaN codes, and pages that no request holds NaN scales."""

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


def check(**kw):
    a = Attn(**kw)
    a.run()
    assert bn.spec_get_status() == 0
    a.check()
    return a


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,R", [(1, 1, 1), (4, 4, 1), (8, 2, 1), (4, 2, 8), (7, 1, 3), (6, 2, 11),
                                      (4, 1, 16), (2, 2, 65), (12, 3, 40)])
def test_head_layouts_and_rows(dtype, d, Hq, Hkv, R):
    check(seed=Hq * 100 + R, Hq=Hq, Hkv=Hkv, R=R, d=d, S=(213, 40), dtype=dtype, mask="tree")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 112, 128, 240, 256])
def test_page_sizes(ps, d):
    check(seed=ps, B=5, S=(0, 1, ps, 2 * ps + 1, 3 * ps - 1), ps=ps, R=5, d=d, mask="chain")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("S", [(0,), (1,), (15,), (16,), (127,), (128,), (129,), (255,), (257,),
                               (2000,)])
def test_lengths(S, dtype):
    check(seed=S[0], B=1, S=S, R=3, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_soft,R,S", [(1, 4, (0, 5)), (16, 20, (300, 129)), (64, 70, (90, 0)),
                                        (63, 256, (17, 200)), (5, 1, (64, 64))])
def test_soft_prompt(dtype, n_soft, R, S):
    check(seed=n_soft, Hq=4, Hkv=2, R=R, S=S, n_soft=n_soft, dtype=dtype, mask="tree")


@pytest.mark.parametrize("R,G", [(120, 4), (256, 1), (60, 8), (33, 3)])
def test_many_rows(R, G):
    check(seed=R, B=3, Hq=2 * G, Hkv=2, R=R, S=(700, 0, 130), mask="tree", n_soft=16)


def test_single_token_decode_of_a_ragged_batch():
    check(seed=9, B=40, Hq=8, Hkv=2, R=1, mask="chain", pad=False,
          S=np.random.default_rng(1).integers(0, 900, 40))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q_scale", [1e-3, 8.0, 60.0])
def test_flat_and_sharp_scores(q_scale, dtype):
    check(seed=3, B=3, Hq=8, Hkv=2, R=9, S=(1500, 800, 64), q_scale=q_scale, mask="chain", dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_explicit_scale_and_splits(dtype):
    check(seed=4, S=(1000, 300), scale=0.31, split=64, dtype=dtype)
    check(seed=4, S=(1000, 300), scale=0.31, split=512, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["wide", "odd", "one_large", "zero_block"])
def test_scales_of_blocks(kind, dtype):
    """Scales that differ by many powers of two between pages, that are no
    powers of two, one page far above the others, and a block of zeros with
    the least scale."""
    rng = np.random.default_rng(8)

    def scale(shape):
        s = 2.0 ** rng.integers(-9, -6, size=shape)
        if kind == "wide":
            s[..., 1] = 2.0 ** rng.integers(-24, 4, size=shape[:2])
        elif kind == "odd":
            s = s * rng.uniform(1, 2, size=shape)
        elif kind == "one_large":
            s[shape[0] // 2, :, 1] = 64.0
        else:
            s[::2, :, 1] = 2.0 ** -60
        return s
    check(seed=5, B=3, Hq=4, Hkv=2, R=6, S=(400, 150, 16), kv_scale=scale, dtype=dtype, mask="chain")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    a = Attn(seed=6, B=2, R=6, S=(0, 50), dtype=dtype, pad=False)
    # request 0 has no prefix: a valid row without any visible column (as a
    # padding row for the oracle, which takes no softmax over nothing)
    a.valid[0, 2] = a.vis[0, 2] = False
    a.words[0, 2] = 0
    a.d_vis.copy_(torch.from_numpy(a.words))
    a.valid[1, 3] = False                  # and a padding row over a prefix
    a.vis[1, 3] = False
    a.d_flags[1, 3] = 0
    a.run()
    assert bn.spec_get_status() == 0
    assert torch.all(a.o[0, 2] == 0) and torch.all(a.lse[0, :, 2] == -float("inf"))
    assert torch.all(a.o[1, 3] == 0) and torch.all(a.lse[1, :, 3] == -float("inf"))
    a.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("x", [0, 1])
def test_a_nan_block_makes_its_readers_nan_and_no_others(dtype, x):
    a = Attn(seed=7, B=3, Hq=4, Hkv=2, R=5, S=(200, 90, 300), dtype=dtype)
    want = Attn(seed=7, B=3, Hq=4, Hkv=2, R=5, S=(200, 90, 300), dtype=dtype)
    want.run()
    a.d_scales[int(a.table[0, 3]), 1, x] = float("nan")
    a.run()
    assert bn.spec_get_status() == 0
    o, l = a.o.float(), a.lse
    assert torch.isnan(o[0, :, 2:]).all()
    if x == 0:
        assert torch.isnan(l[0, 2:]).all()
    else:                                  # the scores are the keys' alone
        assert torch.allclose(l[0], want.lse[0], rtol=2.0 ** -20, atol=1e-6)
    assert torch.equal(o[0, :, :2], want.o[0, :, :2].float()) and torch.equal(l[0, :2], want.lse[0, :2])
    assert torch.equal(o[1:], want.o[1:].float()) and torch.equal(l[1:], want.lse[1:])


def test_non_finite_queries_stay_in_their_rows():
    a = Attn(seed=10, B=2, Hq=4, Hkv=2, R=5, S=(200, 90))
    want = Attn(seed=10, B=2, Hq=4, Hkv=2, R=5, S=(200, 90))
    want.run()
    a.d_q[0, 1, 2, 5] = float("nan")
    a.d_q[1, 0, 0, 3] = float("inf")
    a.run()
    assert torch.isnan(a.o[0, 1, 2]).all() and torch.isnan(a.o[1, 0, 0]).all()
    keep = torch.ones_like(a.o, dtype=torch.bool)
    keep[0, 1, 2] = keep[1, 0, 0] = False
    assert torch.equal(a.o[keep], want.o[keep])


def test_repeated_calls_are_bit_identical():
    a = check(seed=11, B=4, Hq=8, Hkv=2, R=8, S=(900, 100, 2500, 0))
    o, l = a.o.clone(), a.lse.clone()
    for _ in range(3):
        a.ws.fill_(0xFF)
        a.run()
        assert torch.equal(a.o, o) and torch.equal(a.lse, l)


def test_a_call_on_another_stream_and_in_a_graph():
    a = Attn(seed=12, B=3, Hq=8, Hkv=2, R=8, S=(900, 100, 1500))
    a.run()
    torch.cuda.synchronize()
    o, l = a.o.clone(), a.lse.clone()
    s = torch.cuda.Stream()
    a.o.zero_()
    s.wait_stream(torch.cuda.current_stream())
    a.run(stream=s)
    s.synchronize()
    assert torch.equal(a.o, o) and torch.equal(a.lse, l)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    for _ in range(2):
        a.o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.o, o) and torch.equal(a.lse, l)
    assert bn.spec_get_status() == 0


def test_two_calls_at_once_with_their_own_workspaces():
    calls = [Attn(seed=20 + i, B=3, Hq=8, Hkv=2, R=8, S=(900, 100, 1500 + 60 * i)) for i in range(2)]
    want = []
    for a in calls:
        a.run()
        torch.cuda.synchronize()
        want.append((a.o.clone(), a.lse.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for a, s in zip(calls, streams):
            s.wait_stream(torch.cuda.current_stream())
            a.run(stream=s)
    torch.cuda.synchronize()
    for a, (o, l) in zip(calls, want):
        assert torch.equal(a.o, o) and torch.equal(a.lse, l)
    assert bn.spec_get_status() == 0


def test_device_errors_are_reported():
    a = Attn(seed=13, B=3, R=4, S=(200, 90, 300))
    a.d_S[1] = 10 ** 8
    a.run()
    assert bn.spec_get_status() & bn.SPEC_DEV_SEQ_OVERFLOW
    a = Attn(seed=13, B=3, R=4, S=(200, 90, 300))
    a.d_table[2, 5] = 10 ** 6
    a.run()
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_PAGE
    # the other requests are as they were
    a.check(requests=[0, 1])


def test_a_cache_of_many_gigabytes():
    """Pages past the 4 GB mark of a 9.7 GB cache (offsets beyond 32 bits)."""
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs a large device")
    a = Attn(seed=14, B=2, Hq=8, Hkv=8, R=2, S=(300, 77), ps=64, d=128)
    n = 74000
    big = torch.zeros((n,) + tuple(a.d_kv.shape[1:]), dtype=torch.uint8, device="cuda")
    scales = torch.full((n, 8, 2), float("nan"), device="cuda")
    P = a.d_kv.shape[0]
    ids = torch.arange(P, device="cuda") * 9001 + 1900
    assert int(ids.max()) < n
    big[ids] = a.d_kv.view(torch.uint8)
    scales[ids] = a.d_scales
    table = torch.where(a.d_table >= 0, a.d_table * 9001 + 1900, a.d_table)
    a.cache = bn.kv8_desc(big, scales, table)
    a.run()
    assert bn.spec_get_status() == 0
    a.check()
