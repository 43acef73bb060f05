"""The 8-bit cache's operators as a serving step uses them: prompts planned and
appended, then verification steps of attention, logits adjustment, vocabulary
reduction, acceptance and commit, eagerly and as one captured graph.  Also the
attention's bounded waits, and what the Python entry points refuse."""

import numpy as np
import pytest
import torch

import gpu_helpers as gh
import oracle
from kv8_helpers import TABLE, Attn, to_storage, torch_dt, unpack
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    gh.require_gpu()
    bn.spec_get_status()


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Server:
    """B requests over one cache: device buffers, and the oracle's state."""

    def __init__(self, seed, dtype, d=128, ps=16, Hq=8, Hkv=2, R=12, V=3001,
                 prompts=(1, 16, 37, 150), capacity=16):
        self.rng = rng = np.random.default_rng(seed)
        B = len(prompts)
        self.shape, self.dtype, self.ps, self.V = (B, R, Hq, Hkv, d), dtype, ps, V
        self.dt = torch_dt(dtype)
        n_pages = B * capacity
        self.free = rng.permutation(n_pages).astype(np.int32)
        self.kv = torch.zeros((n_pages, Hkv, ps // 8, 2, 8, d), dtype=torch.uint8,
                              device="cuda").view(torch.float8_e4m3fn)
        self.scales = torch.ones((n_pages, Hkv, 2), device="cuda")
        self.table, self.head = torch.full((B, capacity), -1, dtype=torch.int32, device="cuda"), i32(1)
        self.d_free, self.seq = dev(self.free), i32(B)
        self.cache = bn.kv8_desc(self.kv, self.scales, self.table)
        # the oracle's cache, as values
        self.o_codes = np.zeros((n_pages, Hkv, 2, ps, d))
        self.o_scales = np.ones((n_pages, Hkv, 2))
        self.o_table, self.o_seq = np.full((B, capacity), -1, dtype=np.int32), np.zeros(B, dtype=np.int32)
        self.o_head = 0
        self.prompts = np.array(prompts, dtype=np.int32)
        # a step's outputs
        self.o = torch.empty((B, R, Hq, d), dtype=self.dt, device="cuda")
        self.lse = torch.empty((B, Hq, R), device="cuda")
        self.attn = bn.attn_desc(B, R, Hq, Hkv, d, bn.spec_dtype(self.o))
        self.ws = torch.empty(bn.spec_verify_attn_kv8_workspace_size(self.attn, self.cache),
                              dtype=torch.uint8, device="cuda")
        self.adjusted = torch.empty((B, R, V), dtype=self.dt, device="cuda")
        self.am, self.zl, self.zp = i32(B, R), torch.empty((B, R), device="cuda"), torch.empty((B, R), device="cuda")
        self.acc, self.path, self.next, self.last = i32(B), i32(B, R), i32(B), i32(B)

    def prefill(self):
        B, R, Hq, Hkv, d = self.shape
        n = int(self.prompts.sum())
        # the rows of a fused projection: K and V inside wider rows
        qkv = to_storage(self.rng.standard_normal((n, Hq + 2 * Hkv, d)), self.dtype)
        x = dev(qkv).to(self.dt)
        cu, slots, new_len = i32(B + 1), torch.empty(n, dtype=torch.int64, device="cuda"), i32(B)
        bn.spec_page_plan(self.ps, self.kv.shape[0], self.seq, dev(self.prompts), self.table, self.d_free,
                          self.head, cu, slots, new_len)
        bn.kv8_append(self.cache, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots)
        self.seq.copy_(new_len)
        t, h, _, s, ln = kv8.page_plan(self.o_seq, self.prompts, self.o_table, self.free, 0, self.ps, n)
        self.o_table, self.o_head, self.o_seq = t, h, ln
        self.o_codes, self.o_scales = kv8.append(self.o_codes, self.o_scales, qkv[:, Hq:Hq + Hkv],
                                                 qkv[:, Hq + Hkv:], s, self.ps)
        self.same_cache()

    def same_cache(self):
        assert np.array_equal(TABLE[unpack(self.kv)], self.o_codes)
        assert np.array_equal(self.scales.double().cpu().numpy(), self.o_scales)
        assert np.array_equal(self.table.cpu().numpy(), self.o_table)
        assert np.array_equal(self.seq.cpu().numpy(), self.o_seq)
        assert int(self.head) == self.o_head

    def draft(self):
        """A step's inputs: a tree, its rows, and logits that follow it for a
        few levels."""
        B, R, Hq, Hkv, d = self.shape
        rng, V = self.rng, self.V
        x = {}
        x["parent"] = np.full((B, R), -1, dtype=np.int32)
        for r in range(1, R):
            x["parent"][:, r] = rng.integers(max(0, r - 4), r, size=B)
        x["tokens"] = rng.integers(0, V, size=(B, R)).astype(np.int32)
        z = rng.standard_normal((B, R, V)) * 2
        for b in range(B):
            for r in range(1, R, 2):
                z[b, x["parent"][b, r], x["tokens"][b, r]] += 12 + r
        x["logits"] = to_storage(z, self.dtype)
        x["hist"] = rng.integers(0, V, size=(B, 64)).astype(np.int32)
        x["hist_len"] = rng.integers(0, 65, size=B).astype(np.int32)
        x["n_prompt"] = (x["hist_len"] // 2).astype(np.int32)
        x["rep"] = rng.uniform(1, 1.3, size=B).astype(np.float32)
        x["pres"] = rng.uniform(0, 0.5, size=B).astype(np.float32)
        x["freq"] = rng.uniform(0, 0.2, size=B).astype(np.float32)
        allowed = rng.random((3, V)) < 0.6
        x["row_mask"] = rng.integers(-1, 3, size=(B, R)).astype(np.int32)
        words = -(-V // 32)
        bits = np.zeros((3, words * 32), dtype=np.uint8)
        bits[:, :V] = allowed
        x["mask_bits"] = np.packbits(bits, axis=1, bitorder="little").view(np.int32)
        x["q"] = to_storage(rng.standard_normal((B, R, Hq, d)), self.dtype)
        x["kb"] = to_storage(rng.standard_normal((B, Hkv, R, d)) * 2, self.dtype)
        x["vb"] = to_storage(rng.standard_normal((B, Hkv, R, d)), self.dtype)
        x["n_nodes"] = np.full(B, R, dtype=np.int32)
        vis, valid, sees = oracle.mask_build(x["parent"].astype(np.int64), np.zeros((B, R), dtype=bool))
        W = -(-R // 32)
        wide = np.zeros((B, R, W * 32), dtype=np.uint8)
        wide[:, :, :R] = vis
        x["vis"] = np.packbits(wide, axis=2, bitorder="little").view(np.int32).reshape(B, R, W)
        x["flags"] = valid.astype(np.uint8)
        floats = ("logits", "q", "kb", "vb")
        on = {k: dev(v).to(self.dt) if k in floats else dev(v) for k, v in x.items()}
        return x, on, (vis, valid, sees, allowed)

    def step(self, t, stream=None):
        B, R, _, _, _ = self.shape
        V = self.V
        bn.spec_verify_attn_kv8(self.attn, t["q"], self.cache, t["kb"], t["vb"], None, None, self.seq, t["vis"],
                                t["flags"], self.o, self.lse, self.ws, stream)
        d = bn.logits_desc(B, R, V, bn.spec_dtype(self.o), R, 64, 0, 3)
        bn.spec_logits_adjust(d, t["logits"], self.adjusted, t["hist"], t["hist_len"], t["n_prompt"],
                              t["tokens"], t["parent"], None, t["rep"], t["pres"], t["freq"], None, None,
                              t["mask_bits"], t["row_mask"], stream)
        bn.spec_vocab_reduce(self.adjusted.view(B * R, V), t["tokens"].view(-1), self.am.view(-1),
                             self.zl.view(-1), self.zp.view(-1), stream)
        acc = bn.accept_desc(bn.SPEC_ACCEPT_GREEDY_TREE, 0.0, B, R, V, bn.spec_dtype(self.o), R, R)
        bn.spec_accept(acc, self.adjusted, t["tokens"], t["parent"], None, t["n_nodes"], self.am, self.zl,
                       self.zp, self.acc, self.path, self.next, self.last, stream)
        bn.kv8_commit(self.cache, t["kb"], t["vb"], self.path, self.acc, self.seq, self.d_free, self.head,
                      stream)

    STATE = ("kv", "scales", "table", "seq", "head")
    OUT = ("o", "lse", "adjusted", "am", "zl", "zp", "acc", "path", "next", "last")

    def save(self, names):
        return {n: getattr(self, n).view(torch.uint8).clone() if n == "kv" else getattr(self, n).clone()
                for n in names}

    def restore(self, saved):
        for n, x in saved.items():
            (getattr(self, n).view(torch.uint8) if n == "kv" else getattr(self, n)).copy_(x)

    def check(self, x, masks):
        """The step against the oracle, whose state it moves on."""
        B, R, Hq, Hkv, d = self.shape
        vis, valid, sees, allowed = masks
        a = Attn.__new__(Attn)
        a.shape, a.dtype, a.scale, a.n_soft = self.shape, self.dtype, 0.0, 0
        a.S, a.table = self.o_seq, self.o_table
        a.codes, a.scales = self.codes_before, self.o_scales
        a.q, a.kb, a.vb, a.soft_k, a.soft_v = x["q"], x["kb"], x["vb"], None, None
        a.vis, a.valid, a.sees, a.o, a.lse = vis, valid, sees, self.o, self.lse
        a.check()
        hist = [x["hist"][b, :x["hist_len"][b]].tolist() for b in range(B)]
        node = np.tile(np.arange(R, dtype=np.int32), (B, 1))
        want = kv8.logits_adjust(x["logits"], hist, x["n_prompt"], x["tokens"], x["parent"], node, x["rep"],
                                 x["pres"], x["freq"], [[] for _ in range(B)], allowed, x["row_mask"])
        got = self.adjusted.double().cpu().numpy()
        fin = np.isfinite(want)
        assert np.array_equal(np.isneginf(got), ~fin)
        # half a step of the output's type; the arithmetic before it: four
        # roundings to fp32 of values below 64
        half = 2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -24
        assert np.all(np.abs(got - want)[fin] <= half * np.abs(want[fin]) + 4 * 64 * 2.0 ** -24)
        am, _, zp = oracle.vocab_reduce(got.reshape(B * R, -1), x["tokens"].reshape(-1))
        assert np.array_equal(self.am.cpu().numpy().reshape(-1), am)
        lens = self.acc.cpu().numpy()
        paths = []
        for b in range(B):
            p = oracle.accept_greedy_tree(x["tokens"][b], x["parent"][b], R, am.reshape(B, R)[b])[0]
            paths.append([int(v) for v in p])
            assert self.path[b, :int(lens[b])].tolist() == paths[b]
        self.o_codes, self.o_scales, self.o_table, self.o_seq, self.o_head = kv8.commit(
            self.o_codes, self.o_scales, self.o_table, self.o_seq, self.free, self.o_head, x["kb"], x["vb"],
            paths, self.ps)
        self.same_cache()
        return max(len(p) for p in paths)


@pytest.mark.parametrize("dtype,d,ps", [("bf16", 128, 16), ("bf16", 64, 48), ("f32", 128, 16)])
def test_steps_of_a_server(dtype, d, ps):
    s = Server(11, dtype, d=d, ps=ps)
    s.prefill()
    longest = 0
    side = torch.cuda.Stream()
    for n in range(3):
        s.codes_before = unpack(s.kv).copy()
        x, t, masks = s.draft()
        before = s.save(s.STATE)
        s.step(t)
        torch.cuda.synchronize()
        assert bn.spec_get_status() == 0
        eager = s.save(s.STATE + s.OUT)
        # the same step captured on another stream, and replayed twice from
        # the state before it
        g = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=side):
            s.step(t)
        for _ in range(2):
            s.restore(before)
            for name in s.OUT:
                getattr(s, name).zero_()
            g.replay()
            torch.cuda.synchronize()
            again = s.save(s.STATE + s.OUT)
            for name in s.STATE + s.OUT:
                if name == "path":               # (entries past acc_len are not written)
                    for b in range(s.shape[0]):
                        m = int(s.acc[b])
                        assert torch.equal(again[name][b, :m], eager[name][b, :m])
                    continue
                assert torch.equal(again[name], eager[name]), name
        assert bn.spec_get_status() == 0
        longest = max(longest, s.check(x, masks))
    assert longest > 2          # (trees were accepted past their roots)


@pytest.mark.parametrize("R", [1, 16])
def test_attention_waits_run_out_and_the_context_recovers(R):
    """Every CTA has more tiles than ring slots, so a producer finds a slot
    still held at its first test, and gives up."""
    c = Attn(31, B=4, Hq=32, Hkv=8, R=R, S=(9000, 8000, 8500, 7000), mask="chain", pad=False)
    bn.spec_set_wait_limit(0)
    try:
        c.run()
        torch.cuda.synchronize()
    finally:
        bn.spec_set_wait_limit(-1)
    status = bn.spec_get_status()
    assert status & bn.SPEC_DEV_TIMEOUT, f"status {status:#x}"
    c.run()
    assert bn.spec_get_status() == 0
    c.check(requests=[0, 3], heads=[0, 31])


def test_what_the_python_entry_points_refuse():
    c = Attn(32, R=4)
    ok = dict(q=c.d_q, kb=c.d_kb, vb=c.d_vb, seq_len=c.d_S, vis=c.d_vis, row_flags=c.d_flags, o=c.o, lse=c.lse,
              workspace=c.ws)

    def attn(**kw):
        a = dict(ok, **kw)
        bn.spec_verify_attn_kv8(c.desc, a["q"], c.cache, a["kb"], a["vb"], None, None, a["seq_len"], a["vis"],
                                a["row_flags"], a["o"], a["lse"], a["workspace"])

    attn()
    for name, x in ok.items():
        if name != "workspace":
            with pytest.raises(ValueError, match=name):
                attn(**{name: x[:1]})
        with pytest.raises(TypeError, match="CUDA"):
            attn(**{name: x.cpu()})
    for name in ("q", "kb", "vb", "o"):
        with pytest.raises(TypeError, match=name):
            attn(**{name: ok[name].float()})
    with pytest.raises(ValueError, match="contiguous"):
        attn(q=torch.empty((2, 4, 128, 4), dtype=torch.bfloat16, device="cuda").transpose(2, 3))
    with pytest.raises(bn.SpecError) as e:
        attn(workspace=c.ws[:c.ws.numel() // 2])
    assert e.value.code == 4

    with pytest.raises(TypeError):
        bn.kv8_desc(c.d_kv, c.d_scales.double(), c.d_table)
    with pytest.raises(ValueError):
        bn.kv8_desc(c.d_kv, c.d_scales[:1], c.d_table)
    with pytest.raises(TypeError):
        bn.kv8_desc(c.d_kv, c.d_scales, c.d_table.long())

    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    k = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError, match="slot_map"):
        bn.kv8_append(c.cache, k, k, slots.int())
    with pytest.raises(TypeError, match="v must be"):
        bn.kv8_append(c.cache, k, k.float(), slots)
    with pytest.raises(ValueError, match="heads"):
        bn.kv8_append(c.cache, k.transpose(0, 1).contiguous().transpose(0, 1), k, slots)
    with pytest.raises(ValueError, match="k must be"):
        bn.kv8_append(c.cache, k[:2], k, slots)

    z = torch.zeros((1, 2, 40), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="out"):
        bn.spec_logits_adjust(bn.logits_desc(1, 2, 40, bn.SPEC_BF16), z, z[:, :1])
    with pytest.raises(TypeError, match="history"):
        bn.spec_logits_adjust(bn.logits_desc(1, 2, 40, bn.SPEC_BF16, 0, 4), z, z)
    with pytest.raises(ValueError, match="cu_new"):
        bn.spec_page_plan(16, 8, c.d_S, c.d_S, c.d_table, i32(4), i32(1), i32(2), slots)
    assert bn.spec_get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("x", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_rows_that_no_row_sees(dtype, x):
    """Padding rows of the block (and the soft prompt, where no row sees it)
    may hold anything: every output keeps its bits."""
    a, b = (Attn(33, B=3, R=20, S=(100, 0, 260), n_soft=5, mask="tree", dtype=dtype) for _ in range(2))
    b.d_flags.copy_(b.d_flags & 1)
    a.d_flags.copy_(a.d_flags & 1)
    off = torch.from_numpy(~b.valid).cuda()
    assert off.any()
    b.d_q[off] = x
    at = off[:, None].expand(3, 2, 20)
    b.d_kb[at] = x
    b.d_vb[at] = x
    b.d_sk.fill_(x)
    b.d_sv.fill_(x)
    a.run()
    b.run()
    assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)
    assert bn.spec_get_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_writers_at_the_end_of_a_cache_of_many_gigabytes(dtype):
    """Offsets past 2^32 bytes: pages at the end of a 6 GB cache."""
    rng = np.random.default_rng(34)
    H, d, ps, n_pages, R = 8, 128, 64, 48000, 5
    kv = torch.empty((n_pages, H, ps // 8, 2, 8, d), dtype=torch.uint8, device="cuda")
    sc = torch.ones((n_pages, H, 2), device="cuda")
    assert kv.numel() > 1 << 32
    last = np.array([n_pages - 1, n_pages - 3], dtype=np.int32)
    tail = kv[-4:]
    tail.zero_()
    codes, scales = np.zeros((4, H, 2, ps, d)), np.ones((4, H, 2))
    dt = torch_dt(dtype)
    k, v = (to_storage(rng.standard_normal((ps + 7, H, d)), dtype) for _ in range(2))
    at = np.concatenate([np.arange(ps) + 3 * ps, np.arange(7) + ps])         # within the last four pages
    slots = at + (n_pages - 4) * ps
    cache = bn.kv8_desc(kv, sc, dev(last.reshape(2, 1)))
    bn.kv8_append(cache, dev(k).to(dt), dev(v).to(dt), dev(slots))
    codes, scales = kv8.append(codes, scales, k, v, at, ps)
    kb, vb = (to_storage(rng.standard_normal((2, H, R, d)) * 3, dtype) for _ in range(2))
    seq, table = np.array([0, 7], dtype=np.int32), np.array([[3], [1]], dtype=np.int32)
    d_seq, head = dev(seq), i32(1)
    # the first request's page is a new one: the last of the cache once more
    bn.kv8_commit(cache, dev(kb).to(dt), dev(vb).to(dt), dev(np.tile(np.arange(R, dtype=np.int32), (2, 1))),
                  dev(np.array([R, R], dtype=np.int32)), d_seq, dev(last[:1]), head)
    assert bn.spec_get_status() == 0
    codes, scales, table, seq, h = kv8.commit(codes, scales, table, seq, np.array([3], dtype=np.int32), 0, kb,
                                              vb, [list(range(R))] * 2, ps)
    assert np.array_equal(TABLE[unpack(tail)], codes)
    assert np.array_equal(sc[-4:].double().cpu().numpy(), scales)
    assert d_seq.tolist() == [R, 7 + R] and int(head) == h == 1
