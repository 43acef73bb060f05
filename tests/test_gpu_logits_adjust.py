"""spec_logits_adjust against the float64 oracle: tokens that repeat in the
history, on the path and in both, biases with equal ids, masks that leave
little or nothing, odd vocabularies and addresses, in place and not."""

import math

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import oracle
from kv8_helpers import to_storage, torch_dt
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class Case:
    def __init__(self, seed, B=2, Rj=4, V=1000, H=50, N=6, nb=8, nm=3, dtype="bf16", vocab_used=None,
                 offset=0):
        rng = np.random.default_rng(seed)
        u = vocab_used or V
        self.shape, self.dtype = (B, Rj, V), dtype
        self.z = to_storage(rng.standard_normal((B, Rj, V)) * 4, dtype)
        self.hist = rng.integers(-1, u, size=(B, max(H, 1))).astype(np.int32)
        self.hl = rng.integers(0, H + 1, size=B).astype(np.int32)
        self.hl[0] = H
        self.np_ = (self.hl * rng.random(B)).astype(np.int32)
        self.tok = rng.integers(0, u, size=(B, max(N, 1))).astype(np.int32)
        self.par = np.full((B, max(N, 1)), -1, dtype=np.int32)
        for c in range(1, N):
            self.par[:, c] = rng.integers(max(-1, c - 3), c, size=B)
        self.node = rng.integers(-1, max(N, 0), size=(B, Rj)).astype(np.int32)
        self.rep = rng.uniform(0.5, 2, size=B).astype(np.float32)
        self.pres = rng.uniform(-1, 1, size=B).astype(np.float32)
        self.freq = rng.uniform(0, 1, size=B).astype(np.float32)
        self.ids = rng.integers(-1, u, size=(B, max(nb, 1))).astype(np.int32)
        if nb > 1:
            self.ids[:, nb // 2:2 * (nb // 2)] = self.ids[:, :nb // 2]      # equal ids
        self.bias = rng.standard_normal((B, max(nb, 1))).astype(np.float32)
        self.masks = rng.random((max(nm, 1), V)) < 0.5
        if nm > 1:
            self.masks[1] = False                        # allows nothing
        if nm > 2:
            self.masks[2] = False
            self.masks[2, V - 1] = True                  # one token
        self.rm = rng.integers(-1, max(nm, 0), size=(B, Rj)).astype(np.int32)
        self.H, self.N, self.nb, self.nm, self.offset = H, N, nb, nm, offset

    def put(self, x):
        """The rows, `offset` elements past a 256-byte boundary."""
        buf = torch.zeros(x.size + 64, dtype=torch_dt(self.dtype), device="cuda")
        t = buf[self.offset:self.offset + x.size].view(x.shape)
        t.copy_(dev(x))
        return t

    def run(self, in_place=False, out_offset=None):
        B, Rj, V = self.shape
        z = self.put(self.z)
        if in_place:
            out = z
        else:
            self.offset, keep = (self.offset if out_offset is None else out_offset), self.offset
            out = self.put(np.full(self.shape, 9, dtype=np.float32))
            self.offset = keep
        words = np.zeros((max(self.nm, 1), (V + 31) // 32 * 32), dtype=np.uint8)
        words[:, :V] = self.masks
        words = np.packbits(words, axis=1, bitorder="little").view(np.int32)
        d = bn.logits_desc(B, Rj, V, bn.spec_dtype(z), self.N, self.H, self.nb, self.nm)
        bn.spec_logits_adjust(d, z, out, dev(self.hist), dev(self.hl), dev(self.np_), dev(self.tok),
                              dev(self.par), dev(self.node), dev(self.rep), dev(self.pres),
                              dev(self.freq), dev(self.ids), dev(self.bias), dev(words), dev(self.rm))
        return out

    def want(self):
        B, Rj, V = self.shape
        hist = [self.hist[b, :self.hl[b]].tolist() if self.H else [] for b in range(B)]
        node = self.node if self.N else np.full((B, Rj), -1)
        bias = [list(zip(self.ids[b].tolist(), self.bias[b].astype(np.float64))) if self.nb else []
                for b in range(B)]
        return kv8.logits_adjust(self.z, hist, self.np_, self.tok, self.par, node,
                                 self.rep.astype(np.float64), self.pres.astype(np.float64),
                                 self.freq.astype(np.float64), bias,
                                 self.masks if self.nm else None, self.rm)

    def check(self, out):
        got, want = out.double().cpu().numpy(), self.want()
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        fin = np.isfinite(want)
        # at most 8 + nb fp32 roundings of terms no larger than |z| + |want| +
        # 2 + H + sum |bias|, then the storage's own
        size = np.abs(self.z) * 2 + 3 + self.H + self.N + 4 * self.nb
        tol = (8 + self.nb) * 2.0 ** -24 * size
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        err = np.abs(np.where(fin, got - np.where(fin, want, 0), 0))
        bound = tol + half * np.abs(np.where(fin, want, 0))
        assert np.all(err <= bound), (err - bound).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [
    dict(), dict(V=1), dict(V=7, H=300, vocab_used=5), dict(V=2047), dict(V=2049, vocab_used=60, H=900),
    dict(V=32000, Rj=8, H=4096, vocab_used=300), dict(B=1, Rj=1, V=50272, N=2), dict(H=0), dict(N=0),
    dict(nb=0), dict(nm=0), dict(H=0, N=0, nb=0, nm=0), dict(nb=1024, vocab_used=200), dict(nm=1),
    dict(N=256, Rj=70, vocab_used=40, V=3001), dict(B=5, Rj=33, V=4099, N=33)])
def test_adjust(kw, dtype):
    c = Case(seed=len(str(kw)), dtype=dtype, **kw)
    c.check(c.run())
    c.check(c.run(in_place=True))
    assert bn.spec_get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,out_off", [(1, 1), (3, 3), (0, 1), (5, 2)])
def test_rows_off_16_byte_boundaries(dtype, off, out_off):
    c = Case(seed=off, V=4097, offset=off, dtype=dtype)
    c.check(c.run(out_offset=out_off))
    c.check(c.run(in_place=True))


def test_a_chain_and_identity_rows():
    """Every row follows the node of its number; a chain of equal tokens."""
    c = Case(seed=3, Rj=8, N=8, V=500)
    c.par[:] = np.arange(8) - 1
    c.tok[:] = 17
    c.node[:] = np.arange(8)
    c.check(c.run())
    z, out = dev(c.z).bfloat16(), torch.empty((2, 8, 500), dtype=torch.bfloat16, device="cuda")
    d = bn.logits_desc(2, 8, 500, bn.SPEC_BF16, 8)
    bn.spec_logits_adjust(d, z, out, tokens=dev(c.tok), tree_parent=dev(c.par), frequency=dev(c.freq))
    j = np.arange(1, 9)
    want = c.z[:, :, 17] - c.freq[:, None] * j
    assert np.abs(out[:, :, 17].double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() + 1e-5


def test_no_penalties_copies_and_special_values_pass():
    z = torch.randn(2, 3, 999, device="cuda")
    z[0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0])
    out = torch.zeros_like(z)
    bn.spec_logits_adjust(bn.logits_desc(2, 3, 999, bn.SPEC_F32), z, out)
    assert torch.equal(out.view(torch.int32), z.view(torch.int32))


def test_errors_are_reported_and_left_out():
    def go(change, status, V=300):
        c = Case(seed=4, V=V, nm=2)
        clean = Case(seed=4, V=V, nm=2)
        change(c, clean)
        out = c.run()
        assert bn.spec_get_status() == status
        c.want = clean.want
        c.check(out)
    BI, BT = bn.SPEC_DEV_BAD_INDEX, bn.SPEC_DEV_BAD_TREE

    def hist(c, k):
        c.hist[0, 5], k.hist[0, 5] = 300, -1
    go(hist, BI)

    def length(c, k):
        c.hl[0] = 51
    go(length, BI)

    def bias(c, k):
        c.ids[1, 0], k.ids[1, 0] = 10 ** 6, -1
    go(bias, BI)

    def mask(c, k):
        c.rm[0, 1], k.rm[0, 1] = 2, -1
    go(mask, BI)

    def node(c, k):
        c.node[0, 1], k.node[0, 1] = 6, -1
    go(node, BI)

    def parent(c, k):
        c.par[1, 4], k.par[1, 4] = 4, -1
        c.node[1, 2] = k.node[1, 2] = 4
    go(parent, BT)

    def token(c, k):
        c.tok[1, 4], k.tok[1, 4] = 300, -1
        c.node[1, 2] = k.node[1, 2] = 4
    go(token, BI)


@pytest.mark.parametrize("V", [4000, 4001, 32000])
def test_masked_rows_reduce_and_accept(V):
    """Adjusted logits go on to the vocabulary reduction: -inf logits add
    nothing to the LSE, and a row with nothing left is -inf."""
    c = Case(seed=5, Rj=8, V=V, N=8, nm=3)
    c.rm[:] = np.arange(8) % 4 - 1
    out = c.run()
    am = torch.empty((2, 8), dtype=torch.int32, device="cuda")
    lse, zp = (torch.empty((2, 8), device="cuda") for _ in range(2))
    prop = dev(c.tok)
    bn.spec_vocab_reduce(out.view(16, V), prop.view(16), am.view(16), lse.view(16), zp.view(16))
    z = out.double().cpu().numpy().reshape(16, V)
    some = np.isfinite(z).any(1)
    want_am, want_lse, want_zp = oracle.vocab_reduce(z[some], c.tok.reshape(-1)[some])
    got = lse.double().cpu().numpy().reshape(-1)
    assert np.abs(got[some] / want_lse - 1).max() <= 1e-5
    assert np.all(np.isneginf(got[~some]))
    assert am.cpu().numpy().reshape(-1)[some].tolist() == want_am.tolist()
    assert np.array_equal(zp.double().cpu().numpy().reshape(-1)[some], want_zp)
    # a proposal that the mask forbids is never accepted
    acc = bn.accept_desc(bn.SPEC_ACCEPT_THRESH_CHAIN, 1e-30, 2, 8, V, bn.SPEC_BF16, 8, 8)
    i32 = dict(dtype=torch.int32, device="cuda")
    al, nt, ln = (torch.zeros(2, **i32) for _ in range(3))
    path, nn = torch.zeros((2, 8), **i32), torch.full((2,), 8, **i32)
    bn.spec_accept(acc, out, prop, None, None, nn, am, lse, zp, al, path, nt, ln)
    assert bn.spec_get_status() == 0
    with np.errstate(invalid="ignore"):
        p = z[np.arange(16), c.tok.reshape(-1)].reshape(2, 8) - got.reshape(2, 8)
    for b in range(2):
        k = 0
        while k < 8 and p[b, k] >= math.log(1e-30):
            k += 1
        assert int(al[b]) == k


def test_graph_replay():
    c = Case(seed=6, V=5000, Rj=8)
    out = c.run()
    z, o2 = dev(c.z).bfloat16(), torch.empty_like(out)
    d = bn.logits_desc(2, 8, 5000, bn.SPEC_BF16, 6, 50)
    args = [dev(x) for x in (c.hist, c.hl, c.np_, c.tok, c.par, c.node, c.rep, c.pres, c.freq)]
    bn.spec_logits_adjust(d, z, o2, *args)
    want = o2.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bn.spec_logits_adjust(d, z, o2, *args)
    o2.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, want) and bn.spec_get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(B=70, Rj=1, V=20000, H=600, N=2, vocab_used=900),
                                dict(B=90, Rj=3, V=16001, H=900, N=4, nb=300, vocab_used=5000),
                                dict(B=160, Rj=1, V=8197, H=20, N=0, nb=0, nm=1)])
def test_few_rows_of_many_requests(kw, dtype):
    """Decoding batches, whose calls take wider slices of the vocabulary."""
    c = Case(seed=7, dtype=dtype, **kw)
    c.check(c.run())
    c.check(c.run(in_place=True))
    assert bn.spec_get_status() == 0
