"""spec_verify_attn_kv8 on rows whose weights are not flat: one token that
holds most of a row's weight, ahead of a long prefix whose values share a
sign, so that what the small weights add up to is seen."""

import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from kv8_helpers import Attn, pack, to_storage
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def store(a, k, v):
    """Request 0's prefix k, v [Hkv][S][d] into the call's cache: e4m3 codes
    under the least power of two a block allows."""
    ps, S = a.codes.shape[3], int(a.S[0])
    for j in range(-(-S // ps)):
        for x, rows in ((0, k), (1, v)):
            blk = rows[:, j * ps:min(S, (j + 1) * ps)]
            s = 2.0 ** np.ceil(np.log2(np.abs(blk).max((1, 2)) / 448.0))
            c = torch.from_numpy((blk / s[:, None, None]).astype(np.float32)).to(torch.float8_e4m3fn)
            page = a.table[0, j]
            a.codes[page, :, x, :blk.shape[1]] = c.view(torch.uint8).numpy()
            a.scales[page, :, x] = s
    a.d_kv.view(torch.uint8).copy_(pack(a.codes).view(torch.uint8))
    a.d_scales.copy_(dev(a.scales))


def sink_call(seed, S, R, G, d, nats, at, dtype="bf16", ps=256):
    """One request whose token `at` lies `nats` above the others' scores (sd
    0.5): its value 0.05 of theirs, which have a mean of half their sd."""
    a = Attn(seed, B=1, Hq=G, Hkv=1, d=d, R=R, S=(S,), ps=ps, mask="chain", pad=False, dtype=dtype)
    rng = np.random.default_rng(seed + 1)
    u = rng.standard_normal(d)
    u /= np.linalg.norm(u)
    g = 8 * math.sqrt(d / 128)
    a.q = to_storage(g * u + 0.5 * rng.standard_normal(a.q.shape), dtype)
    k = rng.standard_normal((1, S, d)) * 0.5 / math.sqrt((g * g + 0.25 * d) / d)
    k[0, at] = u * nats * math.sqrt(d) / g
    v = rng.standard_normal((1, S, d)) + 0.5 * np.sign(rng.standard_normal(d))
    v[0, at] *= 0.05
    store(a, k, v)
    a.kb, a.vb = a.kb * 0.25, to_storage(a.vb + 0.5, dtype)
    for name in ("q", "kb", "vb"):
        getattr(a, "d_" + name).copy_(dev(getattr(a, name)))
    return a


def bound(a, O, A, v=None):
    """|dO|: the output's rounding, 2^-8 of it (fp32: 2^-24), and what moves a
    weight.  bf16 rows: P is three e5m2 values of 2^-3 each, 2^-9, from an f16
    value, 2^-11; queries and block keys are off by 2^-17.8 of their row's
    largest, ds = 2^-16.8 max|q| sum|k| scale in a score and 2 ds in a weight;
    sums of up to 2^12 steps, 2^-12.  Block values are off by 2^-17.8 of their
    row's largest.  What is lost of weights below 2^-26 of the row's largest
    is at most 2^-35 of it a token: 2^-18 of sum |v| / N here, in the 1e-5."""
    scale = 1 / math.sqrt(a.shape[4])
    big = np.abs(a.q).max() * a.k_abs * scale
    if a.dtype == "f32":
        return 2.0 ** -22 * np.abs(O) + (2 * 2.0 ** -17 * big + 2.0 ** -12) * A + 1e-7
    ds = 2.0 ** -16.8 * big
    assert ds < 2.0 ** -9
    return (2.0 ** -8 * np.abs(O) + (2.0 ** -9 + 2.0 ** -11 + 2.0 ** -12 + 2 * ds) * A +
            2.0 ** -17.8 * (np.abs(a.vb).max() if v is None else v) + 1e-5)


def outputs(a, B):
    """o [B][R][Hq][d] and lse [B][Hq][R] of B requests like the call's one,
    over the same pages: more units than the GPU has SMs, so that a CTA takes
    most of a unit's steps one after the other."""
    _, R, Hq, Hkv, d = a.shape
    many = lambda x: x.expand((B,) + tuple(x.shape[1:])).contiguous()  # noqa: E731
    cache = bn.kv8_desc(a.d_kv, a.d_scales, many(a.d_table))
    desc = bn.attn_desc(B, R, Hq, Hkv, d, bn.spec_dtype(a.d_q))
    ws = torch.empty(bn.spec_verify_attn_kv8_workspace_size(desc, cache), dtype=torch.uint8, device="cuda")
    o, lse = many(a.o), many(a.lse)
    bn.spec_verify_attn_kv8(desc, many(a.d_q), cache, many(a.d_kb), many(a.d_vb), None, None,
                            dev(np.repeat(a.S, B)), many(a.d_vis), many(a.d_flags), o, lse, ws)
    assert bn.spec_get_status() == 0
    return o.double().cpu().numpy(), lse.double().cpu().numpy()


def check(a, B):
    o, lse = outputs(a, B)
    O, L, A = a.oracle()
    over = np.abs(o - O) / bound(a, O, A)
    at = np.unravel_index(over.argmax(), o.shape)
    assert over.max() <= 1, f"O {o[at]} for {O[0][at[1:]]} at {at}: {over.max()} of its bound"
    # a score's error (below 2^-9, as asserted), fp32 sums and a logarithm of up to 16
    assert np.abs(lse - L).max() <= 2.0 ** -9 + 2.0 ** -12


ROWS = [(1, 8), (4, 4), (8, 4), (16, 4)]          # 8, 16, 32 and 64 packed rows


@pytest.mark.parametrize("R,G", ROWS)
@pytest.mark.parametrize("S,nats,at", [(32768, 11.5, 0), (32768, 13.5, 0), (32768, 14.5, 20000),
                                       (131072, 13.8, 0)])
def test_small_weights_beside_a_dominant_token(S, nats, at, R, G):
    check(sink_call(R + S, S, R, G, 128, nats, at), 160)


@pytest.mark.parametrize("R,G", ROWS[1:])
def test_small_weights_of_fp32_rows(R, G):
    check(sink_call(R, 32768, R, G, 128, 13.5, 0, "f32"), 12)


@pytest.mark.parametrize("R,G", ROWS)
def test_small_weights_with_64_head_dimensions(R, G):
    check(sink_call(R, 32768, R, G, 64, 13.5, 0), 160)


@pytest.mark.parametrize("R,G", [(1, 8), (8, 4), (16, 4)])
def test_small_weights_of_a_unit_spread_over_ctas(R, G):
    check(sink_call(R + 1, 32768, R, G, 128, 13.5, 0), 1)


@pytest.mark.parametrize("size", [1e-33, 1e-30, 1e-20, 1e20, 1e37])
@pytest.mark.parametrize("R,G", [(8, 1), (33, 1), (256, 1), (200, 4)])
def test_block_values_of_any_size(R, G, size):
    """Rows over the block alone, whose values are all tiny or all huge: the
    sums stay finite, and values are held to 2^-110 at least."""
    a = Attn(R, B=2, Hq=G, Hkv=1, R=R, S=(0, 0), mask="chain", pad=False)
    a.d_vb.copy_(a.d_vb.double() * size)
    a.vb = a.d_vb.double().cpu().numpy()
    a.run()
    assert bn.spec_get_status() == 0
    O, L, A = a.oracle()
    o = a.o.double().cpu().numpy()
    assert np.all(np.abs(o - O) <= bound(a, O / size, A / size, np.abs(a.vb).max() / size) * size + 2.0 ** -110)
    assert np.abs(a.lse.double().cpu().numpy() - L).max() <= 2.0 ** -9 + 2.0 ** -12


@pytest.mark.parametrize("R,G", ROWS)
@pytest.mark.parametrize("B", [1, 160])
def test_a_nan_value_scale_beside_a_far_larger_score(R, G, B):
    """The block whose value scale is NaN has weights that underflow fp32
    beside the first step's: 0 x NaN is NaN all the same, in a unit that one
    CTA takes whole and in one that is cut."""
    a = sink_call(R, 384, R, G, 128, 160.0, 0, ps=128)
    for page in (1, 2):                      # the second step, and the third
        keep = float(a.d_scales[int(a.table[0, page]), 0, 1])
        a.d_scales[int(a.table[0, page]), 0, 1] = float("nan")
        o, lse = outputs(a, B)
        assert np.isnan(o).all() and np.isfinite(lse).all()
        a.d_scales[int(a.table[0, page]), 0, 1] = keep
    assert np.isfinite(outputs(a, B)[0]).all()
