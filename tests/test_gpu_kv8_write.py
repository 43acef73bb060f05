"""kv8_commit and kv8_append against the oracle: codes, scales and
bookkeeping have to be equal, byte for byte where nothing is written."""

import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import TABLE, pack, page_layout, random_cache, to_storage, torch_dt, unpack
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def rows(rng, shape, dtype):
    """Rows of many sizes, some zero, among them ones that raise a scale."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-8, 9, size=shape[:-1] + (1,))
    x[rng.random(shape[:-1]) < 0.05] = 0.0
    return to_storage(x, dtype)


def same_values(kv, scales, codes, sc):
    for name, got, want in (("codes", TABLE[unpack(kv)], codes),
                            ("scales", scales.double().cpu().numpy(), sc)):
        bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
        at = np.argwhere(bad)[:3].tolist()
        assert not at, f"{name} differ at {at} ({int(bad.sum())} in all)"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,R,cap,ps", [(2, 8, 8, 16), (1, 1, 1, 16), (5, 40, 33, 16), (3, 70, 70, 48),
                                        (2, 256, 200, 256), (32, 4, 4, 32)])
def test_commit(dtype, d, H, R, cap, ps):
    rng = np.random.default_rng(R * 7 + ps)
    B = 6
    S = np.array([0, 1, ps - 1, ps, 2 * ps + 5, 3 * ps], dtype=np.int32)
    maxp = -(-(int(S.max()) + cap) // ps)
    n_pages, table, free = page_layout(rng, S, maxp, ps, 40 + B * (cap // ps + 2))
    codes, scales = random_cache(rng, n_pages, H, ps, d)
    kb, vb = rows(rng, (B, H, R, d), dtype), rows(rng, (B, H, R, d), dtype)
    acc = rng.integers(0, cap + 1, size=B)
    acc[0], acc[-1] = cap, 0
    paths = [sorted(rng.choice(R, size=a, replace=False).tolist()) for a in acc]
    path = np.full((B, cap), 10 ** 6, dtype=np.int32)       # (entries past acc_len are not read)
    for b in range(B):
        path[b, :acc[b]] = paths[b]
    kv, sc = pack(codes), dev(scales)
    tab, seq, fp, fh = dev(table), dev(S), dev(free), dev(np.array([3], dtype=np.int32))
    bn.kv8_commit(bn.kv8_desc(kv, sc, tab), dev(kb).to(torch_dt(dtype)), dev(vb).to(torch_dt(dtype)),
                  dev(path), dev(acc.astype(np.int32)), seq, fp, fh)
    assert bn.spec_get_status() == 0
    c, s, t, l, head = kv8.commit(TABLE[codes], scales.astype(np.float64), table, S, free, 3, kb, vb,
                                  paths, ps)
    same_values(kv, sc, c, s)
    assert np.array_equal(tab.cpu().numpy(), t) and np.array_equal(seq.cpu().numpy(), l)
    assert int(fh) == head


def append_case(rng, B, H, d, ps, dtype, lo=0, hi=150, held_to=40, pad=0):
    new = rng.integers(lo, hi + 1, size=B).astype(np.int32)
    held = rng.integers(0, held_to + 1, size=B).astype(np.int32)
    maxp = max(1, -(-int((held + new).max()) // ps))
    n_pages, table, free = page_layout(rng, held, maxp, ps, int((new // ps + 2).sum()))
    n = int(new.sum())
    _, _, cu, slots, _ = kv8.page_plan(held, new, table, free, 0, ps, n)
    codes, scales = random_cache(rng, n_pages, H, ps, d)
    wide = rows(rng, (n, 2 * H * d + pad), dtype)
    return codes, scales, slots, wide


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,ps,pad", [(4, 2, 128, 16, 0), (1, 1, 64, 16, 64), (9, 3, 64, 32, 8),
                                          (3, 8, 128, 256, 0), (5, 5, 128, 48, 256)])
def test_append(dtype, B, H, d, ps, pad):
    rng = np.random.default_rng(B * 31 + ps)
    codes, scales, slots, wide = append_case(rng, B, H, d, ps, dtype, lo=1, pad=pad)
    slots[rng.random(len(slots)) < 0.03] = -1                # tokens that are not written
    n = len(slots)
    w = dev(wide).to(torch_dt(dtype))
    k = w[:, :H * d].unflatten(1, (H, d))
    v = w[:, H * d:2 * H * d].unflatten(1, (H, d))
    kv, sc = pack(codes), dev(scales)
    bn.kv8_append(bn.kv8_desc(kv, sc), k, v, dev(slots))
    assert bn.spec_get_status() == 0
    c, s = kv8.append(TABLE[codes], scales.astype(np.float64), wide[:, :H * d].reshape(n, H, d),
                      wide[:, H * d:2 * H * d].reshape(n, H, d), slots, ps)
    same_values(kv, sc, c, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_at_the_edges_of_the_types(dtype):
    """Ties, the largest value, values past every scale, subnormals, zeros;
    a non-finite value makes its block's scale NaN, which stays until the page
    is begun again."""
    rng = np.random.default_rng(5)
    H, d, ps = 1, 64, 16
    codes, scales = random_cache(rng, 8, H, ps, d)
    n = 8 * 16
    x = np.zeros((n, H, d), dtype=np.float32)
    mids = (TABLE[:126] + TABLE[1:127]) / 2
    x[0, 0, :63], x[0, 0, 63] = mids[:63], 448
    x[1, 0, :63] = -mids[63:]
    x[16] = 0.0                                              # page 1: zeros alone
    x[32:35] = 1e-38                                         # page 2: below every scale's steps
    x[48, 0, 0], x[48, 0, 1] = 3e38, -1e5                    # page 3: past the largest scale
    x[64, 0, 3] = math.inf                                   # page 4
    x[80, 0, 3], x[81, 0, 4] = math.nan, 5.0                 # page 5
    x[96, 0, :2] = 448 * 2.0 ** -60, 2.0 ** -70              # page 6: the least scale, exactly
    x[112, 0, :2] = np.nextafter(np.float32(448), np.float32(500)), 1
    x = to_storage(x, dtype) if dtype == "f32" else np.where(
        np.isfinite(x), to_storage(np.where(np.isfinite(x), x, 0), dtype), x)
    slots = np.arange(n, dtype=np.int64)
    kv, sc = pack(codes), dev(scales)
    dx = dev(x.astype(np.float32)).to(torch_dt(dtype))
    bn.kv8_append(bn.kv8_desc(kv, sc), dx, dx, dev(slots))
    x = dx.double().cpu().numpy()
    c, s = kv8.append(TABLE[codes], scales.astype(np.float64), x, x, slots, ps)
    same_values(kv, sc, c, s)
    assert np.isnan(s[4:6]).all() and np.isfinite(s[:4]).all()
    # more rows behind half of a NaN page leave it NaN, at offset 0 renew it
    for first, nan in ((8, True), (0, False)):
        y = dev(np.ones((4, H, d), dtype=np.float32)).to(torch_dt(dtype))
        at = np.arange(4, dtype=np.int64) + 4 * ps + first
        bn.kv8_append(bn.kv8_desc(kv, sc), y, y, dev(at))
        c, s = kv8.append(c, s, np.ones((4, H, d)), np.ones((4, H, d)), at, ps)
        same_values(kv, sc, c, s)
        assert np.isnan(s[4, 0, 0]) == nan
    assert bn.spec_get_status() == 0


def small_commit(B=3, free=6, head=0, acc=(2, 2, 2), S=(16, 32, 5), R=4, cap=4):
    rng = np.random.default_rng(6)
    S = np.array(S, dtype=np.int32)
    n_pages, table, fr = page_layout(rng, S, 4, 16, free)
    codes, scales = random_cache(rng, n_pages, 2, 16, 64)
    kb = rows(rng, (B, 2, R, 64), "bf16")
    path = np.tile(np.arange(cap, dtype=np.int32) % R, (B, 1))
    d = dict(kv=pack(codes), sc=dev(scales), tab=dev(table), kb=dev(kb).bfloat16(), path=dev(path),
             acc=dev(np.array(acc, dtype=np.int32)), seq=dev(S), free=dev(fr),
             head=dev(np.array([head], dtype=np.int32)))

    def go():
        bn.kv8_commit(bn.kv8_desc(d["kv"], d["sc"], d["tab"]), d["kb"], d["kb"], d["path"], d["acc"],
                      d["seq"], d["free"], d["head"])
        return bn.spec_get_status()
    before = {k: v.clone() for k, v in d.items()}
    return d, before, go


def bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def unchanged(d, before, names=("kv", "sc", "tab", "seq", "head")):
    return all(torch.equal(bits(d[n]), bits(before[n])) for n in names)


def test_commit_with_a_short_free_list_writes_nothing():
    d, before, go = small_commit(free=1)
    assert go() == bn.SPEC_DEV_CAPACITY and unchanged(d, before)


def test_commit_skips_requests_it_cannot_serve():
    d, before, go = small_commit(S=(62, 32, 5), acc=(3, 9, 2))   # past the table; longer than the path
    assert go() == bn.SPEC_DEV_CAPACITY | bn.SPEC_DEV_BAD_INDEX
    assert d["seq"].tolist() == [62, 32, 7] and int(d["head"]) == 0
    own = [int(x) for x in before["tab"][2][:1]]
    other = [p for p in range(d["kv"].shape[0]) if p not in own]
    assert torch.equal(bits(d["kv"])[other], bits(before["kv"])[other])


def test_commit_with_bad_rows_and_pages():
    d, before, go = small_commit(S=(3, 32, 5))
    d["path"][0, 1] = 99
    assert go() == bn.SPEC_DEV_BAD_INDEX
    p = int(d["tab"][0, 0])
    kv = d["kv"].view(torch.uint8)[p]
    was = before["kv"].view(torch.uint8)[p]
    # token 4 (the bad entry's slot) keeps its codes
    assert torch.equal(kv[:, 0, :, 4], was[:, 0, :, 4])
    d, before, go = small_commit(S=(3, 32, 5))
    d["tab"][0, 0] = 10 ** 6
    assert go() == bn.SPEC_DEV_BAD_PAGE
    d, before, go = small_commit(S=(3, -1, 5))
    assert go() == bn.SPEC_DEV_SEQ_OVERFLOW


def test_append_skips_slots_past_the_cache():
    rng = np.random.default_rng(9)
    codes, scales = random_cache(rng, 3, 2, 16, 64)
    kv, sc = pack(codes), dev(scales)
    x = rows(rng, (5, 2, 64), "bf16")
    slots = np.array([46, 47, 48, 49, 2 ** 40], dtype=np.int64)
    bn.kv8_append(bn.kv8_desc(kv, sc), dev(x).bfloat16(), dev(x).bfloat16(), dev(slots))
    assert bn.spec_get_status() == bn.SPEC_DEV_BAD_PAGE
    c, s = kv8.append(TABLE[codes], scales.astype(np.float64), x[:2], x[:2], slots[:2], 16)
    same_values(kv, sc, c, s)


def test_commit_graph_replay_and_repeat():
    """A captured commit replays to the same cache from the same state."""
    d, before, go = small_commit()
    assert go() == 0
    want = {n: d[n].clone() for n in ("kv", "sc", "tab", "seq", "head")}

    def reset():
        for n in want:
            bits(d[n]).copy_(bits(before[n]))
    g = torch.cuda.CUDAGraph()
    reset()
    cache = bn.kv8_desc(d["kv"], d["sc"], d["tab"])
    with torch.cuda.graph(g):
        bn.kv8_commit(cache, d["kb"], d["kb"], d["path"], d["acc"], d["seq"], d["free"], d["head"])
    for _ in range(2):
        reset()
        g.replay()
        torch.cuda.synchronize()
        assert unchanged(d, want)
    assert bn.spec_get_status() == 0
