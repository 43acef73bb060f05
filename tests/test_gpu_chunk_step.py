"""Prompts in chunks as a server runs them -- pages planned, queries and keys
rotated, keys and values into the cache, the chunk's attention -- eagerly and as
captured graphs, over each cache; and what the entry points promise of streams,
workspaces, waits, large caches and refusals."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
from chunk_helpers import Chunk, dev, rows_of_pages
from kv8_helpers import TABLE, to_storage, torch_dt, unpack
from oracle import chunk, kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Server:
    """B requests over one cache, fed a chunk of projections at a time."""

    def __init__(self, seed, kind, dtype, B=4, Hq=8, Hkv=2, d=64, ps=16, cap=12, room=120):
        self.rng = np.random.default_rng(seed)
        self.kind, self.dtype, self.dt = kind, dtype, torch_dt(dtype)
        self.shape, self.ps, self.room = (B, Hq, Hkv, d), ps, room
        n_pages = B * cap
        self.free = dev(self.rng.permutation(n_pages).astype(np.int32))
        self.table, self.head, self.seq = i32(B, cap), i32(1), i32(B)
        self.n_new, self.cu, self.new_len = i32(B), i32(B + 1), i32(B)
        self.slots = torch.zeros(room, dtype=torch.int64, device="cuda")
        self.x = torch.zeros((room, (Hq + 2 * Hkv) * d), dtype=self.dt, device="cuda")
        self.q = torch.zeros((room, Hq, d), dtype=self.dt, device="cuda")
        self.o, self.lse = torch.zeros_like(self.q), torch.zeros((room, Hq), device="cuda")
        self.desc = bn.chunk_desc(B, room, Hq, Hkv, d, bn.spec_dtype(self.q))
        self.rope = bn.rope_desc(room, Hq, Hkv, d, d, bn.SPEC_ROPE_HALVES, bn.spec_dtype(self.q))
        self.freqs = bn.spec_rope_freqs(d)
        if kind == "kv8":
            self.kv = torch.zeros((n_pages, Hkv, ps // 8, 2, 8, d), dtype=torch.uint8, device="cuda")
            self.scales = torch.ones((n_pages, Hkv, 2), device="cuda")
            self.cache = bn.kv8_desc(self.kv.view(torch.float8_e4m3fn), self.scales, self.table)
            size, self.attend = bn.spec_chunk_attn_kv8_workspace_size, bn.spec_chunk_attn_kv8
        else:
            self.k = torch.full((n_pages, Hkv, d // 64, ps, 64), float("nan"), dtype=self.dt, device="cuda")
            self.v = self.k.clone()
            self.cache = bn.kv_desc_paged(self.k, self.v, self.table)
            size, self.attend = bn.spec_chunk_attn_workspace_size, bn.spec_chunk_attn
        self.ws = torch.empty(size(self.desc, self.cache), dtype=torch.uint8, device="cuda")
        self.done = [[] for _ in range(B)]      # every request's rows so far

    def part(self, lo, H):
        d = self.shape[3]
        return self.x[:, lo * d:(lo + H) * d].unflatten(1, (H, d))

    def calls(self):
        """One chunk: launches alone."""
        B, Hq, Hkv, d = self.shape
        bn.spec_page_plan(self.ps, self.free.numel(), self.seq, self.n_new, self.table, self.free, self.head,
                          self.cu, self.slots, self.new_len)
        k, v = self.part(Hq, Hkv), self.part(Hq + Hkv, Hkv)
        bn.spec_rope(self.rope, self.freqs, self.part(0, Hq), self.q, k, k, seq_len=self.seq, cu_new=self.cu)
        (bn.kv8_append if self.kind == "kv8" else bn.kv_append)(self.cache, k, v, self.slots)
        self.attend(self.desc, self.q, self.cache, self.seq, self.cu, self.o, self.lse, self.ws)
        self.seq.copy_(self.new_len)

    def feed(self, new):
        """Lengths and projections of the next chunk."""
        rows = to_storage(self.rng.standard_normal(tuple(self.x.shape)), self.dtype)
        self.new, self.rows = np.array(new), rows
        self.n_new.copy_(dev(np.array(new, np.int32)))
        self.x.copy_(dev(rows).to(self.dt))

    def check(self):
        """The chunk's attention against the oracle on what the cache holds, and the
        cache's rows against the rotated projections."""
        B, Hq, Hkv, d = self.shape
        assert bn.spec_get_status() == 0
        held = np.array([len(r) for r in self.done])
        cu = np.concatenate([[0], np.cumsum(self.new)])
        n = int(cu[-1])
        assert np.array_equal(self.cu.cpu().numpy(), cu)
        assert np.array_equal(self.seq.cpu().numpy(), held + self.new)
        pos = np.concatenate([h + np.arange(m) for h, m in zip(held, self.new)])
        freqs = chunk.rope_freqs(d, 10000.0)
        x = self.rows[:n].reshape(n, -1, d)
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -22
        for got, lo, H in ((self.q[:n], 0, Hq), (self.part(Hq, Hkv)[:n], Hq, Hkv)):
            want = chunk.rope(x[:, lo:lo + H], pos, freqs, "halves")
            e = np.abs(got.double().cpu().numpy() - want)
            assert (e <= half * np.abs(want) + 25 * 2.0 ** -24 * np.abs(x).max()).all()
        k = self.part(Hq, Hkv)[:n].double().cpu().numpy()
        for b in range(B):
            for i in range(self.new[b]):
                self.done[b].append((k[cu[b] + i], x[cu[b] + i, Hq + Hkv:].astype(np.float64)))
        table = self.table.cpu().numpy()
        keys, values = [], []
        for b in range(B):
            S = len(self.done[b])
            if self.kind == "kv8":
                ids = table[b, :-(-S // self.ps)]
                val = TABLE[unpack(self.kv.view(torch.float8_e4m3fn))] * self.scales.double().cpu().numpy()[..., None, None]
                both = val[ids].transpose(2, 1, 0, 3, 4).reshape(2, Hkv, -1, d)[:, :, :S]
                keys.append(both[0])
                values.append(both[1])
            else:
                keys.append(rows_of_pages(self.k.double().cpu().numpy(), table[b], S))
                values.append(rows_of_pages(self.v.double().cpu().numpy(), table[b], S))
            if S:
                wk, wv = (np.stack([r[i] for r in self.done[b]], 1) for i in (0, 1))
                tol = 0.0 if self.kind != "kv8" else 2.0 ** -4     # (e4m3, scales that may have grown since)
                for got, want in ((keys[b], wk), (values[b], wv)):
                    assert (np.abs(got - want) <= tol * np.abs(want) + tol * 0.25).all()
        q = self.q.double().cpu().numpy()
        ref = chunk.chunk_attention(q[:n], keys, values, held, cu)
        O, L, A, big = ref
        eps = 2.0 ** -24
        ds = (2 * d + 12) * eps * big
        rel = 2 * ds + 2.0 ** -21 + 2 * (int((held + self.new).max()) + 16) * eps
        out = eps
        if self.dtype == "bf16":
            rel, out = rel + 2.0 ** -8, 2.0 ** -8
        got = self.o[:n].double().cpu().numpy()
        assert (np.abs(got - O) <= rel[..., None] * A * (1 + out) + out * np.abs(O) + 1e-30).all()
        lse = self.lse[:n].double().cpu().numpy()
        assert (np.abs(lse - L) <= ds + 2.0 ** -20 + 300 * eps + 8 * eps * np.abs(L)).all()


CHUNKS = [(40, 1, 0, 33), (1, 1, 70, 1), (1, 20, 1, 1), (0, 0, 0, 1), (30, 60, 1, 29)]


@pytest.mark.parametrize("kind", ["paged", "kv8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_in_turn(kind, dtype):
    s = Server(1, kind, dtype)
    for new in CHUNKS:
        s.feed(new)
        s.calls()
        s.check()


@pytest.mark.parametrize("kind", ["paged", "kv8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_same_as_a_captured_graph(kind, dtype):
    """One graph, replayed with other lengths and rows: what the eager calls give, bit
    for bit."""
    a, b = Server(2, kind, dtype), Server(2, kind, dtype)
    b.feed((1, 0, 2, 1))                                     # (loads the kernels)
    b.calls()
    torch.cuda.synchronize()
    b = Server(2, kind, dtype)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.calls()
    for new in CHUNKS:
        a.feed(new)
        a.calls()
        b.feed(new)
        g.replay()
        n = sum(new)
        assert torch.equal(a.o[:n], b.o[:n]) and torch.equal(a.lse[:n], b.lse[:n])
        assert torch.equal(a.seq, b.seq) and torch.equal(a.table, b.table)
    assert bn.spec_get_status() == 0


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_with_workspaces_of_their_own(kind, dtype):
    cs = [Chunk(20 + i, kind, dtype, 128, 8, 2, (200, 1, 3), (300, 900, 0)) for i in range(2)]
    for c in cs:
        c.run()
    torch.cuda.synchronize()
    want = [(c.o.clone(), c.lse.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for c in cs:
        c.o.fill_(3.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st in zip(cs, streams):
            c.run(st)
    torch.cuda.synchronize()
    for c, (o, lse) in zip(cs, want):
        n = int(c.cu[-1])
        assert torch.equal(c.o[:n], o[:n]) and torch.equal(c.lse, lse)
        assert (c.o[n:] == 3.0).all()                         # (rows of no request)


def double_attention(c, rows):
    """o, lse and sum w|v| of some rows in 64 bits, by torch on the GPU."""
    B, n, Hq, Hkv, d = c.shape
    G = Hq // Hkv
    out = []
    for row in rows:
        b = int(np.searchsorted(c.cu, row, side="right")) - 1
        seen = int(c.held[b]) + row - int(c.cu[b]) + 1
        k, v = (torch.from_numpy(np.ascontiguousarray(x[b][:, :seen])).cuda().double() for x in (c.k, c.v))
        q = c.d_q[row].double().view(Hkv, G, d)
        s = torch.einsum("hgd,htd->hgt", q, k) / d ** 0.5
        lse = torch.logsumexp(s, 2)
        w = torch.exp(s - lse[..., None])
        big = torch.einsum("hgd,htd->hgt", q.abs(), k.abs()).amax(2) / d ** 0.5
        out.append([torch.einsum("hgt,htd->hgd", w, x).reshape(Hq, d).cpu().numpy() for x in (v, v.abs())]
                   + [lse.reshape(Hq).cpu().numpy(), big.reshape(Hq).cpu().numpy()])
    return [np.stack(x) for x in zip(*out)]


@pytest.mark.parametrize("kind,ps", [("paged", 16), ("paged", 64), ("contiguous", 0), ("kv8", 64)])
@pytest.mark.parametrize("new,held,Hq,Hkv", [
    ((700, 900), (3000, 0), 8, 8),              # parts of many steps: the rings go round
    ((1,) * 60, (2100,) * 60, 16, 4),           # two-head units, many parts
    ((1, 20, 700, 1, 31), (4000, 2000, 100, 0, 777), 20, 5)])     # an odd head over
def test_many_steps_a_part(kind, ps, new, held, Hq, Hkv):
    c = Chunk(31, kind, "bf16", 128, Hq, Hkv, new, held, ps=ps or 16)
    c.run()
    assert bn.spec_get_status() == 0
    rng = np.random.default_rng(0)
    n = int(c.cu[-1])
    rows = np.unique(np.concatenate([c.cu[:-1], c.cu[1:] - 1, rng.integers(0, n, 40)]))
    O, A, L, big = double_attention(c, rows)
    to, tl = c.tolerance(O, L, A, big)
    got, lse = c.o.double().cpu().numpy(), c.lse.double().cpu().numpy()
    assert np.isfinite(got[:n]).all() and np.isfinite(lse[:n]).all()
    assert (np.abs(got[rows] - O) <= to).all() and (np.abs(lse[rows] - L) <= tl).all()
    assert np.linalg.norm(got[rows] - O) <= 2.0 ** -8 * np.linalg.norm(O)
    o, lse = c.o.clone(), c.lse.clone()
    for _ in range(20):
        c.run()
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("kind", ["paged", "kv8"])
def test_offsets_past_32_bits(kind):
    """A cache of more than 2^32 bytes: pages at its end."""
    Hkv, d, ps = 8, 128, 128
    per = Hkv * d * ps * (2 if kind == "paged" else 2)       # bytes of a page: of k, or of kv
    n_pages = (9 << 29) // per + 3
    c = Chunk(40, kind, "bf16", d, 16, Hkv, (30, 1), (500, 260), ps=ps)
    used = int(c.table[c.table >= 0].max()) + 1
    far = n_pages - used
    if kind == "paged":
        k = torch.full((n_pages, Hkv, d // 64, ps, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = torch.full_like(k, float("nan"))
        k[far:far + c.d_k.shape[0]] = c.d_k[:used] if far + c.d_k.shape[0] > n_pages else c.d_k
        v[far:far + c.d_v.shape[0]] = c.d_v[:used] if far + c.d_v.shape[0] > n_pages else c.d_v
        c.d_table += far
        c.cache = bn.kv_desc_paged(k, v, c.d_table)
    else:
        kv = torch.full((n_pages, Hkv, ps // 8, 2, 8, d), 0x7F, dtype=torch.uint8, device="cuda")
        sc = torch.full((n_pages, Hkv, 2), float("nan"), device="cuda")
        kv[far:] = c.d_kv.view(torch.uint8)[:used]
        sc[far:] = c.d_scales[:used]
        c.d_table += far
        c.cache = bn.kv8_desc(kv.view(torch.float8_e4m3fn), sc, c.d_table)
    c.run()
    assert bn.spec_get_status() == 0
    c.check()


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
def test_results_on_16_byte_boundaries(kind):
    """o and q 16 bytes off a larger boundary."""
    c = Chunk(50, kind, "bf16", 128, 8, 2, (40, 5), (100, 30))
    flat = torch.full((c.o.numel() + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(c.d_q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    q[8:] = c.d_q.reshape(-1)
    c.o, c.d_q = flat[8:].view(c.o.shape), q[8:].view(c.o.shape)
    c.run()
    c.check()


@pytest.mark.parametrize("kind", ["paged", "contiguous", "kv8"])
@pytest.mark.parametrize("new,held", [((400, 300), (2000, 0)), ((1,) * 20, (3000,) * 20)])
def test_waits_run_out(kind, new, held):
    """With no patience every wait that is not met at once gives up: the status says
    so, and the next call is right."""
    c = Chunk(60, kind, "bf16", 128, 8, 4, new, held)
    c.run()
    assert bn.spec_get_status() == 0
    o, lse = c.o.clone(), c.lse.clone()
    old = bn.spec_set_wait_limit(0)
    try:
        c.run()
        assert bn.spec_get_status() & bn.SPEC_DEV_TIMEOUT
    finally:
        bn.spec_set_wait_limit(-1)
    c.run()
    assert bn.spec_get_status() == 0
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    assert old > 0


@pytest.mark.parametrize("kind", ["paged", "kv8"])
def test_refusals_of_chunk_attention(kind):
    c = Chunk(70, kind, "bf16", 64, 4, 2, (3, 4), (5, 6))
    args = dict(q=c.d_q, seq=c.d_seq, cu=c.d_cu, o=c.o, lse=c.lse, ws=c.ws, cache=c.cache)

    def call(**kw):
        a = dict(args, **kw)
        c.call(c.desc, a["q"], a["cache"], a["seq"], a["cu"], a["o"], a["lse"], a["ws"])

    for kw, err in [(dict(q=c.d_q.float()), TypeError), (dict(q=c.d_q[:5]), ValueError),
                    (dict(q=c.d_q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                    (dict(q=c.d_q.cpu()), TypeError), (dict(o=c.o[:, :2]), ValueError),
                    (dict(o=c.o.float()), TypeError), (dict(lse=c.lse.double()), TypeError),
                    (dict(lse=c.lse.T), ValueError), (dict(seq=c.d_seq.long()), TypeError),
                    (dict(seq=c.d_seq[:1]), ValueError), (dict(cu=c.d_cu[:2]), ValueError), (dict(cu=None), TypeError),
                    (dict(ws=c.ws[:100]), bn.SpecError), (dict(ws=c.ws[16:]), bn.SpecError),
                    (dict(o=c.d_q), bn.SpecError)]:
        with pytest.raises(err):
            call(**kw)
    assert bn.spec_get_status() == 0


def test_refusals_of_rope_and_append():
    q, k = torch.zeros(6, 4, 64, device="cuda"), torch.zeros(6, 2, 64, device="cuda")
    d, f = bn.rope_desc(6, 4, 2, 64, 64, 0, bn.SPEC_F32), bn.spec_rope_freqs(64)
    pos = i32(6)
    for args, kw, err in [
            ((d, f, q, q, k, k), dict(), TypeError), ((d, f, q, q, k, k), dict(positions=pos.long()), TypeError),
            ((d, f, q, q, k, k), dict(positions=pos[:5]), ValueError),
            ((d, f, q, q, k, k), dict(seq_len=i32(2)), TypeError),
            ((d, f, q, q, k, k), dict(seq_len=i32(2), cu_new=i32(2)), ValueError),
            ((d, [0.1] * 31, q, q, k, k), dict(positions=pos), ValueError),
            ((d, f, q.half(), q, k, k), dict(positions=pos), TypeError),
            ((d, f, q, q, None, None), dict(positions=pos), TypeError),
            ((d, f, q, q[:, :2], k, k), dict(positions=pos), ValueError),
            ((d, f, q, q, k, q[:, :2]), dict(positions=pos), bn.SpecError),
            ((d, [float("nan")] * 32, q, q, k, k), dict(positions=pos), bn.SpecError)]:
        with pytest.raises(err):
            bn.spec_rope(*args, **kw)
    kc = torch.zeros(2, 2, 16, 64, device="cuda")
    c, slots = bn.kv_desc_contiguous(kc, kc.clone()), torch.zeros(6, dtype=torch.int64, device="cuda")
    for args, err in [((k.bfloat16(), k, slots), TypeError), ((k, k[:, :1], slots), ValueError),
                      ((k, k, slots.int()), TypeError), ((k, k, slots[:5]), ValueError), ((k.cpu(), k, slots), TypeError),
                      ((k.transpose(0, 1).contiguous().transpose(0, 1), k, slots), ValueError)]:
        with pytest.raises(err):
            bn.kv_append(c, *args)
    assert bn.spec_get_status() == 0


def test_a_cache_of_another_device_is_refused():
    x = torch.zeros(2, 2, 16, 64, device="cuda")
    p = torch.zeros(2, 2, 1, 16, 64, device="cuda")
    rows, slots = torch.zeros(6, 2, 64, device="cuda"), torch.zeros(6, dtype=torch.int64, device="cuda")
    o, lse, ws = torch.zeros_like(rows), torch.zeros(6, 2, device="cuda"), torch.zeros(1 << 20, device="cuda")
    d = bn.chunk_desc(1, 6, 2, 2, 64, bn.SPEC_F32)
    for cache in (bn.kv_desc_contiguous(x, x.clone()), bn.kv_desc_paged(p, p.clone(), i32(1, 2))):
        assert cache.device == torch.cuda.current_device()
        cache.device += 1
        with pytest.raises(ValueError):
            bn.kv_append(cache, rows, rows, slots)
        with pytest.raises(ValueError):
            bn.spec_chunk_attn(d, rows, cache, i32(1), i32(2), o, lse, ws)
    assert bn.spec_get_status() == 0
