"""Inputs and comparisons of the chunk operators' tests."""

import numpy as np
import torch

from kv8_helpers import NAN_CODE, TABLE, pack, page_layout, random_cache, to_storage, torch_dt
from oracle import chunk
from self_speculative_verification_gb300 import binding as bn


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def rows_of_pages(x, table, S):
    """Paged rows [P][H][d / 64][ps][64] -> [H][S][d] of one request."""
    ps = x.shape[3]
    ids = table[:-(-S // ps)]
    y = x[ids].transpose(1, 0, 3, 2, 4)                     # [H][page][ps][d / 64][64]
    return y.reshape(y.shape[0], -1, y.shape[3] * 64)[:, :S]


class Chunk:
    """One chunk attention call: inputs on the device, and the oracle's outputs.
    kind: "paged", "contiguous" or "kv8".  Places that no row may use hold NaN."""

    def __init__(self, seed, kind="paged", dtype="bf16", d=128, Hq=8, Hkv=2, new=(5, 1, 0, 130),
                 held=(100, 0, 7, 33), ps=16, q_scale=1.0, scale=0.0, kv_scale=None, tail=3, wide=0,
                 cap=None):
        rng = np.random.default_rng(seed)
        new, held = np.array(new, dtype=np.int32), np.array(held, dtype=np.int32)
        B, n, total = len(new), int(new.sum()) + tail, held + new
        self.new, self.held, self.kind, self.dtype, self.scale = new, held, kind, dtype, scale
        self.shape = (B, n, Hq, Hkv, d)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.q = to_storage(rng.standard_normal((n, Hq, d)) * q_scale, dtype)
        dt = torch_dt(dtype)
        # rows of q lie inside wider ones
        q = torch.full((n, Hq * d + wide), float("nan"), dtype=dt, device="cuda")
        q[:, :Hq * d] = dev(self.q).to(dt).view(n, Hq * d)
        self.d_q = q[:, :Hq * d].unflatten(1, (Hq, d))
        self.k, self.v = [], []
        if kind == "contiguous":
            longest = max(1, int(total.max()) + (cap or 0))
            k = to_storage(rng.standard_normal((B, Hkv, longest, d)), dtype)
            v = to_storage(rng.standard_normal((B, Hkv, longest, d)), dtype)
            for b in range(B):
                k[b, :, total[b]:], v[b, :, total[b]:] = np.nan, np.nan
                self.k.append(k[b, :, :total[b]])
                self.v.append(v[b, :, :total[b]])
            self.d_k, self.d_v = dev(k).to(dt), dev(v).to(dt)
            self.cache = bn.kv_desc_contiguous(self.d_k, self.d_v)
        else:
            cap = cap or max(1, -(-int(total.max()) // ps))
            n_pages, self.table, _ = page_layout(rng, total, cap, ps, 2)
            self.d_table = dev(self.table)
            used = np.zeros((n_pages, ps), dtype=bool)
            for b in range(B):
                for t in range(int(total[b])):
                    used[self.table[b, t // ps], t % ps] = True
        if kind == "paged":
            shape = (n_pages, Hkv, d // 64, ps, 64)
            k, v = (to_storage(rng.standard_normal(shape), dtype) for _ in range(2))
            for b in range(B):
                self.k.append(rows_of_pages(k, self.table[b], total[b]))
                self.v.append(rows_of_pages(v, self.table[b], total[b]))
            hide = ~np.broadcast_to(used[:, None, None, :, None], shape)
            k, v = np.where(hide, np.nan, k), np.where(hide, np.nan, v)
            self.d_k, self.d_v = dev(k.astype(np.float32)).to(dt), dev(v.astype(np.float32)).to(dt)
            self.cache = bn.kv_desc_paged(self.d_k, self.d_v, self.d_table)
        if kind == "kv8":
            codes, scales = random_cache(rng, n_pages, Hkv, ps, d, kv_scale)
            val = TABLE[codes] * scales[..., None, None].astype(np.float64)
            for b in range(B):
                ids = self.table[b, :-(-int(total[b]) // ps)]
                x = val[ids].transpose(2, 1, 0, 3, 4).reshape(2, Hkv, -1, d)[:, :, :total[b]]
                self.k.append(x[0])
                self.v.append(x[1])
            codes = np.where(used[:, None, None, :, None], codes, NAN_CODE).astype(np.uint8)
            scales = np.where(used.any(1)[:, None, None], scales, np.nan).astype(np.float32)
            self.codes, self.scales = codes, scales
            self.d_kv, self.d_scales = pack(codes), dev(scales)
            self.cache = bn.kv8_desc(self.d_kv, self.d_scales, self.d_table)
        self.d_seq, self.d_cu = dev(held), dev(self.cu)
        self.o = torch.full((n, Hq, d), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((n, Hq), 7.0, dtype=torch.float32, device="cuda")
        self.desc = bn.chunk_desc(B, n, Hq, Hkv, d, bn.spec_dtype(self.o), scale)
        self.size, self.call = ((bn.spec_chunk_attn_kv8_workspace_size, bn.spec_chunk_attn_kv8)
                                if kind == "kv8" else
                                (bn.spec_chunk_attn_workspace_size, bn.spec_chunk_attn))
        self.ws = torch.full((self.size(self.desc, self.cache),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        self.call(self.desc, self.d_q, self.cache, self.d_seq, self.d_cu, self.o, self.lse, self.ws,
                  stream)

    def oracle(self):
        return chunk.chunk_attention(self.q, self.k, self.v, self.held, self.cu, self.scale)

    def tolerance(self, O, L, A, big):
        """Elementwise bounds on |dO| and |dLSE|, eps = 2^-24.

        Scores: d products and sums in fp32, each off by eps of the sum of
        |q||k| so far (the tensor cores cut where fp32 rounds: twice that), and
        two more for the scale and the reference: ds = (2 d + 8) eps big.  A
        score's error moves its weight by e^ds against a sum that moves as much:
        2 ds.  exp2 is good to 2^-21, its argument, at most 2 big log2(e) away
        from 0, is rounded once more, which counts as 4 eps big.  Sums over L
        weights in fp32: (L + 16) eps of the sum of their magnitudes, in O and
        in the sum they are divided by.  bf16 rows: a weight is rounded to bf16,
        2^-8 of itself, and so is the result.  8-bit caches with scales that are
        no powers of two: keys and values are rounded to bf16 as well, which
        moves a score by 2^-8 big."""
        eps, n_seen = 2.0 ** -24, float((self.held + self.new).max())
        ds = (2 * self.shape[4] + 12) * eps * big
        odd = (self.kind == "kv8" and self.dtype == "bf16" and
               bool((np.frexp(self.scales[np.isfinite(self.scales)])[0] != 0.5).any()))
        if odd:
            ds = ds + 2.0 ** -8 * big
        rel = 2 * ds + 2.0 ** -21 + 2 * (n_seen + 16) * eps
        out = eps
        if self.dtype == "bf16":
            rel, out = rel + 2.0 ** -8 + (2.0 ** -8 if odd else 0.0), 2.0 ** -8
        to = rel[..., None] * A * (1 + out) + out * np.abs(O) + 1e-30
        tl = ds + 2.0 ** -21 + (n_seen + 16) * eps + 4 * eps * np.abs(np.where(np.isfinite(L), L, 0.0)) + 4 * eps
        return to, tl

    def check(self, ref=None):
        O, L, A, big = ref or self.oracle()
        got, lse = self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()
        n = int(self.cu[-1])
        assert (got[n:] == 7.0).all() and (lse[n:] == 7.0).all(), "rows behind the last token"
        O, L, A, big, got, lse = O[:n], L[:n], A[:n], big[:n], got[:n], lse[:n]
        to, tl = self.tolerance(O, L, A, big)
        fin = np.isfinite(O)
        assert np.array_equal(np.isfinite(got), fin), "finite where the definition is"
        over = np.abs(got - O)[fin] / to[fin]
        assert over.max(initial=0) <= 1, f"O off by {over.max()} of its bound"
        lf = np.isfinite(L)
        assert np.array_equal(np.isfinite(lse), lf)
        assert np.array_equal(np.isneginf(lse), np.isneginf(L))
        e = np.abs(lse - L)[lf] / tl[lf]
        assert e.max(initial=0) <= 1, f"LSE off by {e.max()} of its bound"
        if self.dtype == "bf16" and fin.all() and O.size > 4096:
            # roundings are independent: two of at most 2^-8 / sqrt(3) in the
            # root mean square of weights and results
            assert np.linalg.norm(got - O) <= 2.0 ** -8 * np.linalg.norm(O)
