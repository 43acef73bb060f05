"""spec_rope against the float64 oracle."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import dev
from kv8_helpers import to_storage, torch_dt
from oracle import chunk
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu
LAYOUT = {"pairs": bn.SPEC_ROPE_PAIRS, "halves": bn.SPEC_ROPE_HALVES}


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def bound(x, want, dtype, attention, positions, freqs):
    """|x|, |y| at most big: the angle is off by a float's rounding of a half
    turn and of the fraction, pi 2^-24; sin and cos by 2^-22 (two units) and the
    factor's rounding, 2^-24; three operations of 2^-24 each: in all 2 big
    attention (pi 2^-24 + 2^-22 + 5 2^-24) <= 25 2^-24 big attention, and the
    result's rounding.  Both sides' 64-bit frequencies (three units) and the
    oracle's angle (one) are rounded, which counts as many positions over: 4
    2^-53 of the angle."""
    big = np.abs(x).max(axis=-1, keepdims=True)
    turn = 2 * 4 * 2.0 ** -53 * np.maximum(np.asarray(positions, np.float64), 0) * max(abs(f) for f in freqs)
    return ((25 * 2.0 ** -24 + turn[:, None, None]) * big * abs(attention)
            + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(want))


def check(got, x, positions, freqs, layout, dtype, attention=1.0):
    want = chunk.rope(x, positions, freqs, layout, attention)
    got = got.double().cpu().numpy()
    rot = 2 * len(freqs)
    assert np.array_equal(got[..., rot:], x[..., rot:].astype(np.float64))      # copied
    e = np.abs(got - want) / (bound(x, want, dtype, attention, positions, freqs) + 1e-300)
    assert e.max(initial=0) <= 1, f"off by {e.max()} of its bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("d,rot", [(128, 128), (64, 32), (80, 80), (80, 26), (256, 256), (8, 2), (64, 62),
                                   (128, 48), (256, 2)])
@pytest.mark.parametrize("Hq,Hk", [(4, 2), (1, 0), (0, 3)])
def test_given_positions(dtype, layout, d, rot, Hq, Hk):
    rng = np.random.default_rng(d + rot + Hq)
    n = 37
    pos = rng.integers(0, 200000, size=n).astype(np.int32)
    pos[:4] = [0, 1, 2 ** 31 - 1, 999983]
    freqs = chunk.rope_freqs(rot, 10000.0)
    dt = torch_dt(dtype)
    qx, kx = (to_storage(rng.standard_normal((n, H, d)), dtype) for H in (Hq, Hk))
    q, k = dev(qx).to(dt), dev(kx).to(dt)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    bn.spec_rope(bn.rope_desc(n, Hq, Hk, d, rot, LAYOUT[layout], bn.spec_dtype(q)),
                 bn.spec_rope_freqs(rot), q, qo, k, ko, positions=dev(pos))
    assert bn.spec_get_status() == 0
    check(qo, qx, pos, freqs, layout, dtype)
    check(ko, kx, pos, freqs, layout, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("rot", [64, 38])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_batch_of_a_joint_projection(dtype, layout, rot, in_place):
    """Positions from lengths, q and k side by side in the same rows, in place too;
    rows of no request stay as they are."""
    rng = np.random.default_rng(rot)
    Hq, Hk, d, new, held = 5, 2, 64, [3, 0, 40, 1], [0, 9, 100000, 77]
    n = sum(new) + 4
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    x = to_storage(rng.standard_normal((n, (Hq + 2 * Hk) * d)), dtype)
    t = dev(x).to(torch_dt(dtype))
    out = t if in_place else torch.full_like(t, 7.0)
    part = lambda y, lo, H: y[:, lo * d:(lo + H) * d].unflatten(1, (H, d))  # noqa: E731
    kind = dict(scaling=bn.SPEC_ROPE_RAMP, factor=4.0, trained_len=2048, low=1.0, high=8.0)
    bn.spec_rope(bn.rope_desc(n, Hq, Hk, d, rot, LAYOUT[layout], bn.spec_dtype(t), 1.25),
                 bn.spec_rope_freqs(rot, 50000.0, **kind), part(t, 0, Hq), part(out, 0, Hq),
                 part(t, Hq, Hk), part(out, Hq, Hk), seq_len=dev(np.array(held, np.int32)), cu_new=dev(cu))
    assert bn.spec_get_status() == 0
    freqs = chunk.rope_freqs(rot, 50000.0, "ramp", 4.0, 2048, 1.0, 8.0)
    pos = np.concatenate([h + np.arange(m) for h, m in zip(held, new)])
    m = len(pos)
    check(part(out, 0, Hq)[:m], x[:m, :Hq * d].reshape(m, Hq, d), pos, freqs,
          layout, dtype, 1.25)
    check(part(out, Hq, Hk)[:m], x[:m, Hq * d:(Hq + Hk) * d].reshape(m, Hk, d), pos, freqs, layout, dtype, 1.25)
    rest = out.float().cpu().numpy()
    stays = x if in_place else np.full_like(x, 7.0)
    assert np.array_equal(rest[m:], stays[m:])
    assert np.array_equal(rest[:, (Hq + Hk) * d:], stays[:, (Hq + Hk) * d:])


def test_negative_positions_stay():
    x = np.random.default_rng(1).standard_normal((6, 2, 64)).astype(np.float32)
    pos = np.array([5, -1, 0, -2 ** 31, 7, -1], dtype=np.int32)
    q = dev(x)
    out = torch.full_like(q, 7.0)
    bn.spec_rope(bn.rope_desc(6, 2, 0, 64, 64, bn.SPEC_ROPE_HALVES, bn.SPEC_F32), bn.spec_rope_freqs(64), q, out,
                 positions=dev(pos))
    got = out.cpu().numpy()
    assert (got[pos < 0] == 7.0).all()
    check(out[dev(pos) >= 0], x[pos >= 0], pos[pos >= 0], chunk.rope_freqs(64, 10000.0), "halves", "f32")


def test_any_frequencies():
    """Negative, zero, and faster than a turn a position."""
    x = np.random.default_rng(2).standard_normal((9, 1, 16)).astype(np.float32)
    f = [0.0, -0.3, 100.0, 1e-300, -1e-20, 6.283185307179586, 3.0, -7.5]
    pos = np.arange(9, dtype=np.int32) * 1001
    q = dev(x)
    out = torch.empty_like(q)
    bn.spec_rope(bn.rope_desc(9, 1, 0, 16, 16, bn.SPEC_ROPE_PAIRS, bn.SPEC_F32), f, q, out, positions=dev(pos))
    check(out, x, pos, f, "pairs", "f32")


def test_what_does_not_turn_passes_as_it_is():
    """Infinities and NaN behind rot_dim do not reach the others, nor change."""
    for layout in (bn.SPEC_ROPE_PAIRS, bn.SPEC_ROPE_HALVES):
        x = torch.randn(5, 3, 64, device="cuda").bfloat16()
        x[..., 20] = float("nan")
        x[..., 21], x[..., 63] = float("inf"), float("-inf")
        out = torch.empty_like(x)
        bn.spec_rope(bn.rope_desc(5, 3, 0, 64, 20, layout, bn.SPEC_BF16), bn.spec_rope_freqs(20), x, out,
                     positions=torch.arange(5, dtype=torch.int32, device="cuda"))
        assert torch.equal(out[..., 20:].view(torch.int16), x[..., 20:].view(torch.int16))
        assert torch.isfinite(out[..., :20]).all()


def test_bad_lengths():
    x = torch.randn(8, 1, 64, device="cuda")
    d = bn.rope_desc(8, 1, 0, 64, 64, bn.SPEC_ROPE_PAIRS, bn.SPEC_F32)
    f = bn.spec_rope_freqs(64)
    i = lambda *a: dev(np.array(a, np.int32))  # noqa: E731
    out = torch.full_like(x, 7.0)
    bn.spec_rope(d, f, x, out, seq_len=i(3, -4), cu_new=i(0, 5, 8))
    assert bn.spec_get_status() == bn.SPEC_DEV_SEQ_OVERFLOW
    assert (out[5:] == 7.0).all()
    check(out[:5], x[:5].cpu().numpy(), 3 + np.arange(5), chunk.rope_freqs(64, 10000.0), "pairs", "f32")
    for cu in ((0, 5, 4), (0, 5, 9), (-1, 5, 8)):
        bn.spec_rope(d, f, x, out, seq_len=i(3, 4), cu_new=i(*cu))
        assert bn.spec_get_status() & bn.SPEC_DEV_BAD_INDEX
    # a length at the end of its range: positions go on in 64 bits
    bn.spec_rope(d, f, x, out, seq_len=i(2 ** 31 - 1), cu_new=i(0, 8))
    assert bn.spec_get_status() == 0
    check(out, x.cpu().numpy(), 2 ** 31 - 1 + np.arange(8), chunk.rope_freqs(64, 10000.0), "pairs", "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_rows(dtype):
    """Several tokens a CTA, a last one of fewer."""
    rng = np.random.default_rng(3)
    n, Hq, Hk, d = 20011, 3, 1, 64
    pos = rng.integers(0, 10 ** 6, size=n).astype(np.int32)
    dt = torch_dt(dtype)
    q, k = (torch.randn(n, H, d, device="cuda").to(dt) for H in (Hq, Hk))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    bn.spec_rope(bn.rope_desc(n, Hq, Hk, d, d, bn.SPEC_ROPE_HALVES, bn.spec_dtype(q)), bn.spec_rope_freqs(d), q,
                 qo, k, ko, positions=dev(pos))
    pick = np.concatenate([np.arange(40), rng.integers(0, n, 200), np.arange(n - 40, n)])
    i = dev(pick)
    for x, y in ((q, qo), (k, ko)):
        check(y[i], x[i].double().cpu().numpy(), pos[pick], chunk.rope_freqs(d, 10000.0), "halves", dtype)
