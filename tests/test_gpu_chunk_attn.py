"""spec_chunk_attn and spec_chunk_attn_kv8 against the float64 oracle."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import Chunk, dev
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu

CACHES = [("paged", 16), ("paged", 48), ("paged", 128), ("contiguous", 0), ("kv8", 16), ("kv8", 48),
          ("kv8", 256)]


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def run(c):
    c.run()
    assert bn.spec_get_status() == 0
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,ps", CACHES)
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 4, 4), (128, 7, 1), (64, 10, 2)])
def test_ragged_batch(dtype, kind, ps, d, Hq, Hkv):
    run(Chunk(ps + Hq, kind, dtype, d, Hq, Hkv, ps=ps or 16)).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("new,held", [
    ((1,), (0,)), ((1,), (1,)), ((1, 1, 1), (15, 16, 17)), ((1,), (1500,)), ((2, 1), (127, 128)),
    ((16, 15, 17), (0, 1, 0)), ((128,), (0,)), ((129, 127), (1, 128)), ((64, 65, 63), (64, 63, 65)),
    ((300,), (0,)), ((0, 0, 3, 0), (5, 0, 0, 1 << 20)), ((1,) * 40, tuple(range(40)))])
def test_lengths(dtype, kind, new, held):
    held = tuple(0 if h > 10 ** 5 else h for h in held)
    run(Chunk(len(new) + sum(new), kind, dtype, 128, 8, 2, new, held)).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "kv8"])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 16, 33, 100, 128])
def test_heads_that_share_keys(dtype, kind, G):
    run(Chunk(G, kind, dtype, 64, G, 1, (7, 1, 40), (3, 200, 0))).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("q_scale,scale", [(8.0, 0.0), (1.0, 0.7), (0.0, 0.0), (40.0, 0.0)])
def test_sharp_and_flat_scores(dtype, kind, q_scale, scale):
    run(Chunk(3, kind, dtype, 128, 4, 2, (40, 200), (500, 0), q_scale=q_scale, scale=scale)).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scales_of_any_kind(dtype):
    """Finite scales that the writers do not give."""
    draw = np.random.default_rng(1)
    c = Chunk(4, "kv8", dtype, 128, 8, 2, (5, 100), (60, 10),
              kv_scale=lambda sh: draw.uniform(0.002, 0.02, size=sh))
    run(c).check()


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_are_bit_identical(kind, dtype):
    c = run(Chunk(5, kind, dtype, 128, 8, 2, (3, 200, 1, 1), (700, 40, 1000, 3)))
    o, lse = c.o.clone(), c.lse.clone()
    for fill in (0x00, 0x7F):
        c.ws.fill_(fill)
        c.o.fill_(7.0)
        c.lse.fill_(7.0)
        run(c)
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "contiguous"])
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
def test_non_finite_values_reach_the_rows_that_see_them(dtype, kind, what):
    """A non-finite value in the chunk itself and one in the history of another
    request: rows that do not see it are as if it were not there."""
    c = Chunk(6, kind, dtype, 128, 4, 2, (150, 20, 3), (10, 300, 50))
    places = [(0, 1, 10 + 70, 5), (1, 0, 40, 100)]           # request, head, token, dimension
    for b, h, t, x in places:
        c.v[b][h, t, x] = what
        if kind == "paged":
            c.d_v[c.table[b, t // 16], h, x // 64, t % 16, x % 64] = what
        else:
            c.d_v[b, h, t, x] = what
    run(c)
    O, L, A, big = c.oracle()
    hit = np.zeros(O.shape[:2], dtype=bool)
    for b, h, t, x in places:
        for i in range(int(c.new[b])):
            if c.held[b] + i >= t:
                hit[c.cu[b] + i, 2 * h:2 * h + 2] = True
                got = c.o[int(c.cu[b]) + i, 2 * h:2 * h + 2, x]
                assert not torch.isfinite(got).any()
    got = c.o.double().cpu().numpy()
    n = int(c.cu[-1])
    to, tl = c.tolerance(O[:n], L[:n], A[:n], big[:n])
    ok = ~hit[:n]
    assert (np.abs(got[:n] - O[:n])[ok] <= to[ok]).all()
    lse = c.lse.double().cpu().numpy()[:n]
    assert (np.abs(lse - L[:n]) <= tl).all()                  # (values do not reach it)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_non_finite_keys_and_queries(dtype, what):
    c = Chunk(7, "paged", dtype, 128, 4, 2, (150, 20, 3), (10, 300, 50))
    t = 10 + 40
    c.k[0][1, t, 3] = what
    c.d_k[c.table[0, t // 16], 1, 0, t % 16, 3] = what
    c.q[int(c.cu[1]) + 4, 0, 7] = what
    c.d_q[int(c.cu[1]) + 4, 0, 7] = what
    run(c)
    O, L, A, big = c.oracle()
    # (infinities: a score of either sign, which the definition settles)
    n = int(c.cu[-1])
    got, lse = c.o.double().cpu().numpy()[:n], c.lse.double().cpu().numpy()[:n]
    assert np.array_equal(np.isnan(got), np.isnan(O[:n])) and np.array_equal(np.isnan(lse), np.isnan(L[:n]))
    fin = np.isfinite(O[:n])
    assert fin.any() and (~fin).any()
    to, tl = c.tolerance(np.nan_to_num(O[:n]), L[:n], np.nan_to_num(A[:n]), big[:n])
    assert (np.abs(got - O[:n])[fin] <= to[fin]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_blocks_with_nan_scales(dtype):
    """A key block of NaN scale, seen: o = lse = NaN; a value block: o = NaN."""
    c = Chunk(8, "kv8", dtype, 128, 4, 2, (60, 5), (20, 100))
    c.d_scales[int(c.table[0, 3]), 0, 0] = float("nan")       # tokens 48 .. 63 of request 0, head 0
    c.d_scales[int(c.table[1, 6]), 1, 1] = float("nan")       # tokens 96 .. of request 1, head 1
    run(c)
    O, L, A, big = c.oracle()
    n = int(c.cu[-1])
    o_nan, l_nan = np.zeros((n, 4), dtype=bool), np.zeros((n, 4), dtype=bool)
    o_nan[48 - 20:60, :2] = l_nan[48 - 20:60, :2] = True
    o_nan[60:, 2:] = True
    got, lse = c.o.double().cpu().numpy()[:n], c.lse.double().cpu().numpy()[:n]
    assert np.array_equal(np.isnan(got).all(-1), o_nan) and np.array_equal(np.isnan(got).any(-1), o_nan)
    assert np.array_equal(np.isnan(lse), l_nan)
    to, _ = c.tolerance(O[:n], L[:n], A[:n], big[:n])
    assert (np.abs(got - O[:n])[~o_nan] <= to[~o_nan]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "kv8"])
def test_codes_and_rows_of_wider_rows(dtype, kind):
    """q inside wider rows, whose other elements are NaN."""
    run(Chunk(9, kind, dtype, 64, 6, 3, (9, 33), (4, 70), wide=128)).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
def test_bad_lengths_skip_their_request(dtype, kind):
    c = Chunk(10, kind, dtype, 64, 4, 2, (5, 6, 7), (10, 20, 30))
    O, L, A, big = c.oracle()
    for seq, cu, bits, skipped in [
            ([10, -1, 30], [0, 5, 11, 18], bn.SPEC_DEV_SEQ_OVERFLOW, [1]),
            ([10, 20, 1 << 29], [0, 5, 11, 18], bn.SPEC_DEV_SEQ_OVERFLOW, [2]),
            ([10, 20, 2 ** 31 - 1], [0, 5, 11, 18], bn.SPEC_DEV_SEQ_OVERFLOW, [2]),
            ([10, 20, 30], [0, 5, 11, 1000], bn.SPEC_DEV_BAD_INDEX, [2]),
            ([10, 20, 30], [-3, 5, 11, 18], bn.SPEC_DEV_BAD_INDEX, [0]),
            ([10, 20, 30], [0, 5, 4, 4], bn.SPEC_DEV_BAD_INDEX, [1, 2])]:
        c.d_seq, c.d_cu = dev(np.array(seq, np.int32)), dev(np.array(cu, np.int32))
        c.o.fill_(7.0)
        c.lse.fill_(7.0)
        c.run()
        assert bn.spec_get_status() == bits
        got = c.o.double().cpu().numpy()
        to, _ = c.tolerance(O[:18], L[:18], A[:18], big[:18])
        for b in range(3):
            rows = slice(int(c.cu[b]), int(c.cu[b + 1]))
            if b in skipped:
                assert (got[rows] == 7.0).all()
            else:
                assert (np.abs(got[rows] - O[rows]) <= to[rows]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["paged", "kv8"])
def test_bad_pages_are_not_read(dtype, kind):
    """A page id outside the cache: reported; other requests are not affected."""
    c = Chunk(11, kind, dtype, 128, 4, 2, (5, 60, 7), (100, 20, 30))
    c.d_table[0, 2], c.d_table[0, 3] = -5, 1 << 30
    c.run()
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_PAGE
    O, L, A, big = c.oracle()
    got = c.o.double().cpu().numpy()
    n = int(c.cu[-1])
    to, _ = c.tolerance(O[:n], L[:n], A[:n], big[:n])
    assert (np.abs(got[5:n] - O[5:n]) <= to[5:]).all()


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_requests(kind, dtype):
    """More requests than the kernels have threads."""
    rng = np.random.default_rng(2)
    new, held = rng.integers(0, 3, 1300), rng.integers(0, 40, 1300)
    run(Chunk(12, kind, dtype, 64, 2, 1, new, held)).check()


@pytest.mark.parametrize("kind", ["paged", "kv8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_long_row_over_all_ctas(kind, dtype):
    """A single token behind a long history: its keys are shared out."""
    run(Chunk(13, kind, dtype, 128, 4, 1, (1, 2), (40000, 9), ps=64)).check()


@pytest.mark.parametrize("kind", ["paged", "kv8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ps", [80, 128, 256])
def test_long_pages(kind, dtype, ps):
    """Pages as long as a step or longer, and of a size that does not divide it."""
    run(Chunk(14, kind, dtype, 128, 6, 3, (70, 1, 9, 200), (300, 511, 0, 57), ps=ps)).check()
