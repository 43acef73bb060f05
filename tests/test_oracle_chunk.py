"""Pins of the chunk operators' oracle: library special cases, closed forms,
invariants; and the frequencies that spec_rope_freqs computes on the host."""

import math

import numpy as np
import pytest
import torch

import oracle
from oracle import chunk
from self_speculative_verification_gb300 import binding as bn


@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rope_scores_depend_on_the_distance_alone(layout):
    rng = np.random.default_rng(0)
    f = chunk.rope_freqs(16, 100.0)
    q, k = rng.standard_normal((2, 1, 1, 16))
    at = lambda x, p: chunk.rope(x, [p], f, layout)[0, 0]  # noqa: E731
    for m, n in ((3, 10), (1000, 1007), (50, 57)):
        assert math.isclose(at(q, m) @ at(k, n), at(q, 0) @ at(k, 7), rel_tol=1e-9)
    assert np.array_equal(at(q, 0), q[0, 0])
    assert math.isclose(np.linalg.norm(at(q, 12345)), np.linalg.norm(q), rel_tol=1e-12)


def test_rope_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 12))
    f = chunk.rope_freqs(8, 10.0)
    perm = [0, 2, 4, 6, 1, 3, 5, 7, 8, 9, 10, 11]            # halves <- pairs
    a = chunk.rope(x, [0, 3, 5, 9], f, "pairs", 2.0)[..., perm]
    assert np.allclose(a, chunk.rope(x[..., perm], [0, 3, 5, 9], f, "halves", 2.0), rtol=1e-14, atol=0)
    z = (x[..., 0:8:2] + 1j * x[..., 1:8:2])[3] * 2.0 * np.exp(9j * f)
    y = chunk.rope(x, [0, 3, 5, 9], f, "pairs", 2.0)[3]
    assert np.allclose(y[:, 0:8:2], z.real) and np.allclose(y[:, 1:8:2], z.imag)
    assert np.array_equal(y[:, 8:], x[3, :, 8:])
    assert np.array_equal(chunk.rope(x, [-1] * 4, f, "pairs"), x)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (80, 500000.0), (256, 1e6), (6, 0.5)])
@pytest.mark.parametrize("name,kind,args", [
    ("plain", bn.SPEC_ROPE_PLAIN, {}), ("linear", bn.SPEC_ROPE_LINEAR, dict(factor=8.0)),
    ("ramp", bn.SPEC_ROPE_RAMP, dict(factor=8.0, trained_len=8192.0, low=1.0, high=4.0)),
    ("ramp", bn.SPEC_ROPE_RAMP, dict(factor=0.5, trained_len=100.0, low=0.0, high=32.0))])
def test_frequencies(rot, base, name, kind, args):
    got = np.array(bn.spec_rope_freqs(rot, base, kind, **args))
    want = chunk.rope_freqs(rot, base, name, **args)
    assert got.shape == want.shape and np.allclose(got, want, rtol=1e-14, atol=0)


def test_ramp_by_hand():
    # base 2 pi: pair i of 8 turns once in (2 pi)^(1 + i / 4) positions
    f = chunk.rope_freqs(8, (2 * math.pi) ** 4, "ramp", 4.0, (2 * math.pi) ** 3, 1.0, (2 * math.pi) ** 2)
    plain = (2 * math.pi) ** -np.arange(4.0)
    w = ((2 * math.pi) - 1) / ((2 * math.pi) ** 2 - 1)
    assert np.allclose(f, plain * [1.0, w + (1 - w) / 4, 0.25, 0.25])


@pytest.mark.parametrize("held,new", [((0, 7, 3), (4, 1, 0)), ((9,), (1,))])
def test_attention_is_causal_library_attention(held, new):
    rng = np.random.default_rng(2)
    Hq, Hkv, d = 4, 2, 8
    cu = np.concatenate([[0], np.cumsum(new)])
    q = rng.standard_normal((int(cu[-1]) + 2, Hq, d))
    ks = [rng.standard_normal((Hkv, h + n, d)) for h, n in zip(held, new)]
    vs = [rng.standard_normal((Hkv, h + n, d)) for h, n in zip(held, new)]
    o, lse, mag, big = chunk.chunk_attention(q, ks, vs, held, cu)
    for b in range(len(new)):
        n, S = new[b], held[b]
        if n == 0:
            continue
        t = lambda x: torch.from_numpy(np.repeat(x, Hq // Hkv, axis=0))  # noqa: E731
        rows = torch.from_numpy(q[cu[b]:cu[b + 1]]).transpose(0, 1)
        mask = torch.arange(S + n) <= S + torch.arange(n)[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(rows, t(ks[b]), t(vs[b]), attn_mask=mask)
        assert np.allclose(o[cu[b]:cu[b + 1]], want.transpose(0, 1).numpy())
        s = (rows @ t(ks[b]).transpose(1, 2) / math.sqrt(d)).masked_fill(~mask, -math.inf)
        assert np.allclose(lse[cu[b]:cu[b + 1]], torch.logsumexp(s, 2).T.numpy())
        assert (np.abs(o[cu[b]:cu[b + 1]]) <= mag[cu[b]:cu[b + 1]] + 1e-12).all()
    assert np.isnan(o[cu[-1]:]).all()


def test_attention_agrees_with_the_verification_oracle():
    """A chunk is a chain of speculative rows whose own K/V are in the cache."""
    rng = np.random.default_rng(3)
    n, S, H, d = 5, 11, 2, 16
    q = rng.standard_normal((n, H, d))
    k, v = rng.standard_normal((2, H, S + n, d))
    o, lse, _, _ = chunk.chunk_attention(q, [k], [v], [S], [0, n], 0.3)
    vis, valid, sees = oracle.mask_build(np.arange(n)[None] - 1, np.zeros((1, n), bool))
    O, L = oracle.verify_attention(q[None], [k[:, :S]], [v[:, :S]], k[None, :, S:], v[None, :, S:], vis, valid,
                                   sees, scale=0.3)
    assert np.allclose(o, O[0]) and np.allclose(lse, L[0].T)


def test_attention_of_non_finite_places():
    q, k, v = np.ones((3, 1, 2)), np.ones((1, 3, 2)), np.arange(6.0).reshape(1, 3, 2)
    v[0, 1, 0] = np.nan
    o, lse, _, _ = chunk.chunk_attention(q, [k], [v], [0], [0, 3])
    assert np.isfinite(o[0]).all() and np.isnan(o[1:, 0, 0]).all() and np.isfinite(o[1:, 0, 1]).all()
    assert np.allclose(lse[:, 0], math.sqrt(2) + np.log([1, 2, 3]))
    k[0, 2] = -np.inf                                        # weight 0
    v[0, 1, 0] = 2.0
    o, lse, _, _ = chunk.chunk_attention(q, [k], [v], [0], [0, 3])
    assert np.allclose(o[2, 0], v[0, :2].mean(0))
    o, lse, _, _ = chunk.chunk_attention(q, [np.full((1, 3, 2), -np.inf)], [v], [0], [0, 3])
    assert (o == 0).all() and np.isneginf(lse).all()


def test_append_by_hand():
    kc, vc = np.zeros((2, 1, 1, 16, 64)), np.zeros((2, 1, 1, 16, 64))
    k, v = np.ones((3, 1, 64)), np.full((3, 1, 64), 2.0)
    a, b = chunk.append_rows(kc, vc, k, v, [17, -1, 2], True)
    assert a.sum() == 128 and (a[1, 0, 0, 1] == 1).all() and (b[0, 0, 0, 2] == 2).all() and kc.sum() == 0
    a, _ = chunk.append_rows(np.zeros((2, 1, 5, 64)), np.zeros((2, 1, 5, 64)), k, v, [9, 0, -5], False)
    assert (a[1, 0, 4] == 1).all() and (a[0, 0, 0] == 1).all() and a.sum() == 128
