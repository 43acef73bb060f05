"""Inputs and comparisons of the 8-bit cache's tests."""

import math

import numpy as np
import torch

import oracle
from oracle import kv8
from self_speculative_verification_gb300 import binding as bn
from self_speculative_verification_gb300.workloads import round_bf16

TABLE = kv8.e4m3_table()
NAN_CODE = 0x7F


def to_storage(x, dtype):
    x = np.asarray(x, dtype=np.float32)
    return round_bf16(x) if dtype == "bf16" else x


def torch_dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def pack(codes_u8):
    """uint8 codes [P][H][2][ps][d] -> the cache's [P][H][ps / 8][2][8][d]."""
    P, H, _, ps, d = codes_u8.shape
    x = codes_u8.reshape(P, H, 2, ps // 8, 8, d).transpose(0, 1, 3, 2, 4, 5)
    return torch.from_numpy(np.ascontiguousarray(x)).cuda().view(torch.float8_e4m3fn)


def unpack(kv):
    """The cache's codes as uint8 [P][H][2][ps][d]."""
    x = kv.view(torch.uint8).cpu().numpy()
    P, H, g, _, _, d = x.shape
    return x.transpose(0, 1, 3, 2, 4, 5).reshape(P, H, 2, g * 8, d)


def random_cache(rng, P, H, ps, d, scale=None):
    """Codes (no NaN among them) and scales; scale: None for powers of two
    around 2^-7, or a function of the shape."""
    codes = rng.integers(0, 256, size=(P, H, 2, ps, d)).astype(np.uint8)
    # mostly of ordinary size: exponents 2 .. 13 of 0 .. 15
    codes = (codes & 0x87) | (rng.integers(2, 14, size=codes.shape).astype(np.uint8) << 3)
    codes[rng.random(codes.shape) < 0.02] = 0
    s = 2.0 ** rng.integers(-9, -5, size=(P, H, 2)) if scale is None else scale((P, H, 2))
    return codes, s.astype(np.float32)


def page_layout(rng, held, cap, ps, spare):
    """A shuffled page table for requests of `held` tokens, with -7 in unused
    entries, and the free pages in list order."""
    need = [-(-int(s) // ps) for s in held]
    n_pages = sum(need) + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((len(held), cap), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return n_pages, table, perm[at:].copy()


class Attn:
    """One attention call: inputs on the device, and the oracle's outputs."""

    def __init__(self, seed, B=2, Hq=4, Hkv=2, d=128, R=4, S=(100, 37), ps=16, n_soft=0,
                 dtype="bf16", mask="la", q_scale=1.0, scale=0.0, kv_scale=None, pad=True,
                 split=0, cap=None):
        rng = np.random.default_rng(seed)
        S = np.array(list(S)[:B], dtype=np.int32)
        cap = cap or max(1, -(-int(S.max()) // ps))
        n_pages, table, _ = page_layout(rng, S, cap, ps, 2)
        codes, scales = random_cache(rng, n_pages, Hkv, ps, d, kv_scale)
        used = np.zeros((n_pages, ps), dtype=bool)
        for b in range(B):
            for t in range(int(S[b])):
                used[table[b, t // ps], t % ps] = True
        # slots no token holds are NaN codes, pages nobody holds have NaN scales
        dev_codes = np.where(used[:, None, None, :, None], codes, NAN_CODE).astype(np.uint8)
        dev_scales = np.where(used.any(1)[:, None, None], scales, np.nan).astype(np.float32)
        draw = lambda *sh: to_storage(rng.standard_normal(sh), dtype)  # noqa: E731
        self.q = to_storage(rng.standard_normal((B, R, Hq, d)) * q_scale, dtype)
        self.kb, self.vb = draw(B, Hkv, R, d), draw(B, Hkv, R, d)
        self.soft_k = draw(Hkv, n_soft, d) if n_soft else None
        self.soft_v = draw(Hkv, n_soft, d) if n_soft else None
        par = np.full((B, R), -1, dtype=np.int64)
        if mask == "chain":
            par[:] = np.arange(R) - 1
        elif mask == "tree":
            for r in range(1, R):
                par[:, r] = rng.integers(max(0, r - 7), r, size=B)
        if pad and R > 1:
            par[B - 1, R - max(1, R // 5):] = -2
        self.soft_flags = (rng.random((B, R)) < 0.5) if n_soft else np.zeros((B, R), dtype=bool)
        self.vis, self.valid, self.sees = oracle.mask_build(par, self.soft_flags)
        W = (R + 31) // 32
        bits = np.zeros((B, R, W * 32), dtype=np.uint8)
        bits[:, :, :R] = self.vis
        self.words = np.packbits(bits, axis=2, bitorder="little").view(np.int32).reshape(B, R, W)
        self.shape = (B, R, Hq, Hkv, d)
        self.S, self.table, self.scale = S, table, scale
        self.codes, self.scales, self.dtype = codes, scales, dtype
        dt = torch_dt(dtype)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d_kv, self.d_scales, self.d_table = pack(dev_codes), dev(dev_scales), dev(table)
        self.d_q, self.d_kb, self.d_vb = (dev(x).to(dt) for x in (self.q, self.kb, self.vb))
        self.d_sk = dev(self.soft_k).to(dt) if n_soft else None
        self.d_sv = dev(self.soft_v).to(dt) if n_soft else None
        self.d_S, self.d_vis = dev(S), dev(self.words)
        flags = self.valid * 1 + self.sees * 2
        self.d_flags = dev(flags.astype(np.uint8))
        self.o = torch.full((B, R, Hq, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((B, Hq, R), 7.0, dtype=torch.float32, device="cuda")
        self.cache = bn.kv8_desc(self.d_kv, self.d_scales, self.d_table)
        self.desc = bn.attn_desc(B, R, Hq, Hkv, d, bn.spec_dtype(self.d_q), n_soft, scale, split)
        self.n_soft = n_soft
        n = bn.spec_verify_attn_kv8_workspace_size(self.desc, self.cache)
        self.ws = torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        bn.spec_verify_attn_kv8(self.desc, self.d_q, self.cache, self.d_kb, self.d_vb, self.d_sk,
                                self.d_sv, self.d_S, self.d_vis, self.d_flags, self.o, self.lse,
                                self.ws, stream)

    def oracle(self, requests=None, heads=None):
        """O, LSE and sum p |v| in float64."""
        val = TABLE[self.codes]
        pk, pv = kv8.gather(val, self.scales.astype(np.float64), self.table, self.S)
        args = dict(soft_k=self.soft_k, soft_v=self.soft_v, requests=requests, heads=heads)
        if self.scale:
            args["scale"] = self.scale
        O, L = oracle.verify_attention(self.q, pk, pv, self.kb, self.vb, self.vis, self.valid,
                                       self.sees, **args)
        args["soft_v"] = None if self.soft_v is None else np.abs(self.soft_v)
        A, _ = oracle.verify_attention(self.q, pk, [np.abs(v) for v in pv], self.kb,
                                       np.abs(self.vb), self.vis, self.valid, self.sees, **args)
        # sum |v| over each request's columns, for every query head [B][1][Hq][d]
        v = np.stack([np.abs(x).sum(1) for x in pv]) + np.abs(self.vb).sum(2)
        if self.n_soft:
            v = v + np.abs(self.soft_v).sum(1)
        self.v_sum = np.repeat(v, self.q.shape[2] // v.shape[1], axis=1)[:, None]
        self.k_abs = max([np.abs(k).sum(-1).max() for k in pk if k.size] +
                         [np.abs(self.kb).sum(-1).max()] +
                         ([np.abs(self.soft_k).sum(-1).max()] if self.n_soft else []))
        return O, L, A

    def tolerance(self, O, A, v_sum):
        """Elementwise bounds on |dO| and |dLSE|.

        Scores: bf16 rows reach the tensor cores as the sum of two e4m3
        values with one power-of-two scale a row, so an element is off by at
        most half of e4m3's smallest step, 2^-10, where the row's largest is
        >= 224: 2^-17.8 of it, and a block or soft-prompt key likewise; that
        is ds = 2^-16.8 max|q| sum|k| scale.  fp32 rows: 128 products and sums
        of 2^-24 each, ds = 2^-17 max|q| sum|k| scale at most.  Each moves p
        by a factor within e^(2 ds) and LSE by ds.  P (bf16 rows) is the sum
        of two e4m3 values as well, the second raised by 2^4: it is off by
        2^-8 of itself, or where it is small by half of the raised one's
        smallest step, 2^-14 (or by all of itself, if that is less), under a
        scale that keeps the row's largest P at 2^5 at least.  So a small p is
        off by 2^-19 of the largest, which is at most the sum of all: together
        by 2^-19 sum |v| in O, and by no more than A.  A block or soft-prompt
        value (bf16 rows) is one like a query: off by at most 2^-10 / 224 =
        2^-17.8 of the largest of its row, which the row's weights, whose sum
        is 1, pass on at most whole.  The output's own rounding is 2^-8 (bf16) or 2^-24
        (fp32) of it."""
        B, R, Hq, Hkv, d = self.shape
        scale = self.scale or 1 / math.sqrt(d)
        big = np.abs(self.q).max() * self.k_abs * scale
        if self.dtype == "bf16":
            ds = 2.0 ** -16.8 * big
            v = max([np.abs(self.vb).max()] + ([np.abs(self.soft_v).max()] if self.n_soft else []))
            small = np.minimum(A, 2.0 ** -19 * v_sum)
            return (2.0 ** -8 * np.abs(O) + (2.0 ** -7 + 2 * ds) * A + small + 2.0 ** -17.8 * v + 1e-7,
                    ds + 1e-5)
        ds = 2.0 ** -17 * big
        return 2.0 ** -22 * np.abs(O) + (2 * ds + 2.0 ** -18) * A + 1e-9, ds + 2e-6

    def check(self, requests=None, heads=None):
        B, R, Hq, Hkv, d = self.shape
        O, L, A = self.oracle(requests, heads)
        bs = list(range(B)) if requests is None else list(requests)
        hs = list(range(Hq)) if heads is None else list(heads)
        got = self.o.double().cpu().numpy()[bs][:, :, hs]
        lse = self.lse.double().cpu().numpy()[bs][:, hs]
        O, A, L = O[bs][:, :, hs], A[bs][:, :, hs], L[bs][:, hs]
        to, tl = self.tolerance(O, A, self.v_sum[bs][:, :, hs])
        assert np.isfinite(got).all()
        over = np.abs(got - O) / to
        at = np.unravel_index(over.argmax(), O.shape)
        assert over.max() <= 1, f"O {got[at]} for {O[at]} at {at}: {over.max()} of its bound"
        fin = np.isfinite(L)
        assert np.array_equal(np.isneginf(lse), ~fin)
        if fin.any():
            # (fp32 logarithm and sum: 2^-21 of the value more)
            e = np.abs(lse[fin] - L[fin]) - 2.0 ** -21 * np.abs(L[fin])
            assert e.max() <= tl, f"LSE off by {e.max()}, bound {tl}"
