"""Pins of the 8-bit cache, page plan and logits oracles against something
other than themselves: torch's CPU float8 type, the bf16 commit's oracle,
closed forms and counting."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import kv8


def test_e4m3_table_and_rounding_match_the_cpu_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    t = kv8.e4m3_table()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(codes, nan=1e9))
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 8, 4000),
                        (t[:126] + t[1:127]) / 2, t[:127], -t[:127]])   # ties and values
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv8.round_e4m3(x), want)
    assert kv8.round_e4m3(1e30) == 448 and np.isnan(kv8.round_e4m3(math.inf))


@pytest.mark.parametrize("e", [-61, -60, -9, 0, 3, 59, 60, 61])
def test_block_exponent_is_the_smallest_that_holds_the_value(e):
    top = 448.0 * 2.0 ** e
    clip = lambda v: min(max(v, -60), 60)  # noqa: E731
    assert kv8.block_exponent(top) == clip(e)
    assert kv8.block_exponent(np.nextafter(top, np.inf)) == clip(e + 1)
    assert kv8.block_exponent(0.0) == -60


def test_rows_within_half_a_step_and_growth_is_exact_for_normals():
    rng = np.random.default_rng(2)
    codes = np.zeros((1, 2, 2, 16, 64))
    scales = np.ones((1, 2, 2))
    a = rng.standard_normal((3, 2, 64))
    kv8.write_rows(codes, scales, 0, 0, list(a), list(a))
    val = (codes * scales[..., None, None])[0, :, 0, :3].transpose(1, 0, 2)
    # half a step: 2^-4 of the value, or half the smallest subnormal's step
    assert np.all(np.abs(val - a) <= np.maximum(np.abs(a) * 2.0 ** -4,
                                                scales[0, :, 0][None, :, None] * 2.0 ** -10))
    before = (codes * scales[..., None, None])[0, :, 0, :3].copy()
    big = a[:1] * 64
    kv8.write_rows(codes, scales, 0, 3, list(big), list(big))
    after = (codes * scales[..., None, None])[0, :, 0, :3]
    step = scales[0, :, 0][:, None, None] * 2.0 ** -9
    assert np.all((after == before) | (np.abs(before) < 8 * step))
    assert np.all(np.abs(after - before) <= step / 2)


def test_commit_allocates_as_the_bf16_commit_does():
    rng = np.random.default_rng(3)
    B, H, R, d, ps = 4, 2, 9, 64, 16
    seq = np.array([16, 3, 30, 47], dtype=np.int32)
    table = np.full((B, 5), -9, dtype=np.int32)
    nxt = 0
    for b in range(B):
        for j in range(-(-int(seq[b]) // ps)):
            table[b, j] = nxt
            nxt += 1
    free = np.arange(nxt, nxt + 9, dtype=np.int32)[::-1].copy()
    paths = [[0, 2, 5], [], [1, 3, 4, 8], [7, 8]]
    kb = rng.standard_normal((B, H, R, d))
    pages = np.zeros((nxt + 9, H, 1, ps, 64))
    _, _, pt, s2, head = oracle.kv_commit_paged(pages, pages, table, seq, free, 0, kb, kb, paths, ps)
    codes, scales = np.zeros((nxt + 9, H, 2, ps, d)), np.ones((nxt + 9, H, 2))
    _, _, pt8, s8, head8 = kv8.commit(codes, scales, table, seq, free, 0, kb, kb, paths, ps)
    assert np.array_equal(pt, pt8) and np.array_equal(s2, s8) and head == head8


def test_plan_then_append_is_a_commit_of_all_rows():
    rng = np.random.default_rng(4)
    B, H, d, ps = 3, 2, 64, 16
    seq, new = np.array([5, 0, 32], dtype=np.int32), np.array([20, 16, 1], dtype=np.int32)
    table = np.array([[0, -1, -1], [-1, -1, -1], [1, 2, -1]], dtype=np.int32)
    free = np.array([7, 3, 5, 4, 6], dtype=np.int32)
    codes, scales = np.zeros((8, H, 2, ps, d)), np.ones((8, H, 2))
    rows = rng.standard_normal((B, H, 20, d))
    c1, s1, t1, l1, h1 = kv8.commit(codes, scales, table, seq, free, 0, rows, rows,
                                    [list(range(n)) for n in new], ps)
    t2, h2, cu, slots, l2 = kv8.page_plan(seq, new, table, free, 0, ps, 40)
    packed = np.concatenate([rows[b].transpose(1, 0, 2)[:n] for b, n in enumerate(new)])
    c2, s2 = kv8.append(codes, scales, packed, packed, slots[:37], ps)
    assert np.array_equal(t1, t2) and h1 == h2 and np.array_equal(l1, l2)
    assert np.array_equal(c1, c2) and np.array_equal(s1, s2)
    assert cu.tolist() == [0, 20, 36, 37] and np.all(slots[37:] == -1)
    assert len(set(slots[:37].tolist())) == 37


def test_logits_by_hand():
    z = np.array([[[2.0, -2.0, 1.0, 0.5, 3.0]]])
    out = kv8.logits_adjust(z, [[0, 1, 1]], [1], [[4, 2]], [[-1, 0]], [[1]], [2.0], [0.25], [0.5],
                            [[(3, 1.0), (3, 1.0)]], np.array([[True, True, True, True, False]]), [[0]])
    # 0: prompt only; 1: twice after it; 2 and 4: on the path; 4: masked
    assert out[0, 0].tolist() == [1.0, -5.25, -0.25, 2.5, -math.inf]
