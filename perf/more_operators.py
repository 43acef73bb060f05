"""Cases of a prompt chunk's way through the KV cache: rotary positions of its
queries and keys, its keys and values into the bf16 / fp32 cache, and the
attention of the chunk over that cache or over the 8-bit one.

``own`` False computes each operator in elementary torch operations; ``own``
True makes the library's calls on the same state.  New tokens are packed: token
i of request b is row ``cu_new[b] + i`` and has position ``seq_len[b] + i``.
A paged cache is ``[n_pages][Hkv][head_dim / 64][page_size][64]`` (keys and
values each), a contiguous one ``[B][Hkv][max_seq][head_dim]``; the 8-bit one
holds per (page, KV head) one float8 e4m3 tile ``[page_size / 8][2][8][head_dim]``
and a scale for its keys and one for its values.
"""

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn


def _package():
    from self_speculative_verification_gb300 import binding
    return binding


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # attention, the smallest call: a few new tokens of two requests, fp32
        dict(name="chunk_tiny_f32", op="chunk", B=2, Hq=4, Hkv=2, d=64, lo=1, hi=8, ones=0.0,
             hist_lo=128, hist_hi=200, ps=16, dtype="f32"),
        # a server's mixed batch: most requests decode one token, a few bring a chunk
        dict(name="chunk_mixed", op="chunk", B=48, Hq=32, Hkv=8, d=128, lo=100, hi=512, ones=0.9,
             hist_lo=512, hist_hi=4096, ps=16, dtype="bf16"),
        # whole prompts of a model without shared heads, contiguous cache
        dict(name="chunk_prompts", op="chunk", B=4, Hq=32, Hkv=32, d=128, lo=1024, hi=4096, ones=0.0,
             hist_lo=0, hist_hi=0, ps=0, dtype="bf16"),
        # chunks of long documents behind a long history
        dict(name="chunk_long", op="chunk", B=3, Hq=32, Hkv=8, d=128, lo=512, hi=2048, ones=0.0,
             hist_lo=16384, hist_hi=65536, ps=64, dtype="bf16"),
        # the same over the cache in 8 bits: a small model's short chunks
        dict(name="chunk8_small", op="chunk8", B=8, Hq=8, Hkv=1, d=64, lo=1, hi=40, ones=0.0,
             hist_lo=0, hist_hi=300, ps=16, dtype="bf16"),
        # the mixed batch
        dict(name="chunk8_mixed", op="chunk8", B=48, Hq=32, Hkv=8, d=128, lo=100, hi=512, ones=0.9,
             hist_lo=512, hist_hi=4096, ps=16, dtype="bf16"),
        # the long documents
        dict(name="chunk8_long", op="chunk8", B=3, Hq=32, Hkv=8, d=128, lo=512, hi=2048, ones=0.0,
             hist_lo=16384, hist_hi=65536, ps=64, dtype="bf16"),
        # one chunk of a few prompts enters the cache, fp32
        dict(name="append_chunk_f32", op="append", B=5, Hkv=8, d=128, lo=1, hi=120, held=70, ps=32,
             dtype="f32", pad=0),
        # whole prompts, rows a part of wider projection rows
        dict(name="append_prompts", op="append", B=32, Hkv=8, d=128, lo=100, hi=2048, held=0, ps=16,
             dtype="bf16", pad=4096),
        # the rows of speculative blocks, positions of their own
        dict(name="rope_block", op="rope", B=16, lo=8, hi=8, hist=4096, Hq=32, Hk=32, d=128, rot=128,
             layout="pairs", scaling="plain", given=True, pad=0, dtype="bf16"),
        # a part of each head, positions stretched, fp32
        dict(name="rope_part_f32", op="rope", B=6, lo=100, hi=1500, hist=20000, Hq=8, Hk=2, d=64,
             rot=32, layout="pairs", scaling="linear", given=False, pad=64, dtype="f32"),
        # whole prompts far into a long context, rows of a joint projection
        dict(name="rope_prompts", op="rope", B=32, lo=100, hi=2048, hist=120000, Hq=32, Hk=8, d=128,
             rot=128, layout="halves", scaling="ramp", given=False, pad=1024, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk8", "chunk8", "append", "rope"])
    if op in ("chunk", "chunk8"):
        dtype = rng.choice(["bf16"] * 7 + ["f32"])
        d = rng.choice([64, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8, 32])
        G = rng.choice([1, 2, 4, 5, 7, 8])
        hi = rng.choice([1, _log(rng, 1, 64), _log(rng, 16, 4096), _log(rng, 16, 4096)])
        hist = rng.choice([0, _log(rng, 1, 4096), _log(rng, 64, 65536)])
        most = 2e12 if dtype == "bf16" else 4e10            # (operations)
        while 4 * d * Hkv * G * hi * (hist + hi / 2) > most and hi > 1:
            hi = max(1, hi // 2)
        one = 4 * d * Hkv * G * hi * (hist + hi / 2) + 64 * d * Hkv * (hist + hi)
        B = max(1, min(_log(rng, 1, 64), int(most / one), int(5e8 / ((hist + hi) * Hkv * d))))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, lo=rng.choice([0, 1, (hi + 1) // 2, hi]), hi=hi,
                    ones=rng.choice([0.0, 0.5, 0.9]), hist_lo=rng.choice([0, hist // 2, hist]),
                    hist_hi=hist,
                    ps=rng.choice([16, 32, 48, 64, 128] + ([0, 0] if op == "chunk" else [])),
                    dtype=dtype)
    if op == "append":
        hi = _log(rng, 2, 4096)
        Hkv = rng.choice([1, 4, 8, 32])
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), int(2e5 / (hi * Hkv)))), Hkv=Hkv,
                    d=rng.choice([64, 128]), lo=rng.randint(0, hi // 2), hi=hi,
                    held=rng.choice([0, rng.randint(1, 300)]), ps=rng.choice([0, 16, 32, 48, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 64, 1024]))
    hi = _log(rng, 1, 4096)
    Hq, Hk = rng.choice([(1, 1), (4, 1), (7, 1), (8, 8), (16, 2), (32, 8)])
    d = rng.choice([64, 80, 128, 256])
    return dict(op="rope", B=max(1, min(_log(rng, 1, 64), int(1.6e8 / (hi * (Hq + Hk) * d)))),
                lo=rng.choice([0, 1, hi]), hi=hi, hist=_log(rng, 1, 900000), Hq=Hq, Hk=Hk, d=d,
                rot=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]),
                layout=rng.choice(["pairs", "halves"]),
                scaling=rng.choice(["plain", "linear", "ramp"]), given=rng.choice([True, False]),
                pad=rng.choice([0, 8, 1024]), dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------- the states

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 29)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _new_and_held(case, order=None):
    """New tokens and tokens held, per request: a case has the same ones under
    every seed, in another order."""
    B = case["B"]
    fixed = np.random.default_rng([B, case["lo"], case["hi"]])
    new = fixed.integers(case["lo"], case["hi"] + 1, size=B)
    new[fixed.random(B) < case.get("ones", 0.0)] = 1
    new[0] = case["hi"]
    if case["op"] in ("chunk", "chunk8"):
        held = fixed.integers(case["hist_lo"], case["hist_hi"] + 1, size=B)
        held[0] = case["hist_hi"]
    else:
        held = fixed.integers(0, case["held" if case["op"] == "append" else "hist"] + 1, size=B)
    if order is not None:
        new, held = new[order], held[order]
    return new, held


def prepare(case, seed):
    g, rs = _gen(seed), np.random.default_rng([seed, 7])
    new, held = _new_and_held(case, rs.permutation(case["B"]))
    s = dict(op=case["op"], case=dict(case), new=new.tolist(), held=held.tolist(),
             seq_len=_cuda(held.astype(np.int32)),
             cu_new=_cuda(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)))
    {"chunk": _prepare_chunk, "chunk8": _prepare_chunk, "append": _prepare_append,
     "rope": _prepare_rope}[case["op"]](case, s, g, rs, new, held)
    return s


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _randn(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda").to(dt)


def _pages(rs, tokens, ps, spare):
    """A shuffled page table for requests that hold `tokens`."""
    need = -(-tokens // ps)
    n_pages = int(need.sum()) + spare
    perm = rs.permutation(n_pages).astype(np.int32)
    table = np.zeros((len(tokens), max(1, int(need.max()))), dtype=np.int32)
    table[np.arange(table.shape[1])[None, :] < need[:, None]] = perm[:int(need.sum())]
    return n_pages, table


def _cache_shape(case, n_pages, longest):
    Hkv, d, ps = (case[k] for k in ("Hkv", "d", "ps"))
    return (n_pages, Hkv, d // 64, ps, 64) if ps else (case["B"], Hkv, longest, d)


def _filled(g, shape, dt):
    """Normal values, a part at a time."""
    x = torch.empty(shape, dtype=dt, device="cuda")
    step = max(1, (1 << 28) // max(1, x[0].numel()))
    for i in range(0, shape[0], step):
        x[i:i + step] = torch.randn(x[i:i + step].shape, generator=g, device="cuda")
    return x


def _filled_kv8(g, n_pages, Hkv, ps, d):
    """Blocks of normal keys and values, heads of different sizes."""
    kv = torch.empty((n_pages, Hkv, ps // 8, 2, 8, d), dtype=F8, device="cuda")
    scales = torch.empty((n_pages, Hkv, 2), dtype=torch.float32, device="cuda")
    head = torch.exp2(torch.randint(-2, 3, (1, Hkv, 1, 1, 1, 1), generator=g, device="cuda").float())
    head = torch.cat([torch.ones_like(head), head], 3)                    # (values alone)
    step = max(1, (1 << 27) // (Hkv * ps * 2 * d))
    for i in range(0, n_pages, step):
        x = torch.randn(kv[i:i + step].shape, generator=g, device="cuda") * head
        m, e = torch.frexp(x.abs().amax(dim=(2, 4, 5)))                   # the smallest 2^e that
        s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype))   # holds them
        scales[i:i + step] = s
        kv[i:i + step] = (x / s.view(-1, Hkv, 1, 2, 1, 1)).to(F8)
    return kv, scales


def _prepare_chunk(case, s, g, rs, new, held):
    Hq, Hkv, d, ps, B = (case[k] for k in ("Hq", "Hkv", "d", "ps", "B"))
    dt, n, total = _dt(case), int(new.sum()), held + new
    n_pages = 0
    if ps:
        n_pages, table = _pages(rs, total, ps, 3)
        s["page_table"] = _cuda(table)
    if case["op"] == "chunk8":
        s["kv"], s["scales"] = _filled_kv8(g, n_pages, Hkv, ps, d)
    else:
        shape = _cache_shape(case, n_pages, max(1, int(total.max()) + 5))
        s["k"], s["v"] = _filled(g, shape, dt), _filled(g, shape, dt)
    # heads differ in how sharply they look
    sharp = torch.exp2(torch.rand((1, Hq, 1), generator=g, device="cuda") * 3 - 1)
    s["q"] = (torch.randn((n, Hq, d), generator=g, device="cuda") * sharp).to(dt)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((n, Hq), dtype=torch.float32, device="cuda")
    if own:
        bn = _package()
        s["desc"] = bn.chunk_desc(B, n, Hq, Hkv, d, bn.spec_dtype(s["q"]))
        if case["op"] == "chunk8":
            s["cache"] = bn.kv8_desc(s["kv"], s["scales"], s["page_table"])
            size = bn.spec_chunk_attn_kv8_workspace_size(s["desc"], s["cache"])
        else:
            s["cache"] = (bn.kv_desc_paged(s["k"], s["v"], s["page_table"]) if ps
                          else bn.kv_desc_contiguous(s["k"], s["v"]))
            size = bn.spec_chunk_attn_workspace_size(s["desc"], s["cache"])
        s["workspace"] = torch.empty(max(size, 256), dtype=torch.uint8, device="cuda")


def _prepare_append(case, s, g, rs, new, held):
    B, Hkv, d, ps = (case[k] for k in ("B", "Hkv", "d", "ps"))
    dt, n, total = _dt(case), int(new.sum()), held + new
    b = np.repeat(np.arange(B), new)
    pos = held[b] + np.arange(n) - np.repeat(np.cumsum(new) - new, new)
    n_pages, longest = 0, max(1, int(total.max()) + 3)
    if ps:
        n_pages, table = _pages(rs, total, ps, 3)
        s["page_table"] = _cuda(table)
        slots = table[b, pos // ps].astype(np.int64) * ps + pos % ps
    else:
        slots = b.astype(np.int64) * longest + pos
    shape = _cache_shape(case, n_pages, longest)
    s["k_cache"], s["v_cache"] = _filled(g, shape, dt), _filled(g, shape, dt)
    rows = _randn(g, (n, 2 * Hkv * d + case["pad"]), dt)
    s["k"] = rows[:, :Hkv * d].unflatten(1, (Hkv, d))
    s["v"] = rows[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    s["slot_map"] = _cuda(slots)
    if own:
        bn = _package()
        s["cache"] = (bn.kv_desc_paged(s["k_cache"], s["v_cache"], s["page_table"]) if ps
                      else bn.kv_desc_contiguous(s["k_cache"], s["v_cache"]))


BASE, FACTOR, TRAINED, LOW, HIGH, ATTENTION = 10000.0, 8.0, 4096, 1.0, 4.0, 1.2079


def _freqs(case, pi=math.pi):
    """Radians a position, per pair, in 64 bits: plain, all slowed down by a
    factor, or only those that turn seldom over the trained length."""
    f = BASE ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
    if case["scaling"] == "linear":
        return f / FACTOR
    if case["scaling"] == "ramp":
        w = np.clip((TRAINED * f / (2 * pi) - LOW) / (HIGH - LOW), 0.0, 1.0)
        return f * (w + (1 - w) / FACTOR)
    return f


def _prepare_rope(case, s, g, rs, new, held):
    Hq, Hk, d = (case[k] for k in ("Hq", "Hk", "d"))
    dt, n = _dt(case), int(new.sum())
    rows = _randn(g, (n, (Hq + Hk) * d + case["pad"]), dt)
    s["q"] = rows[:, :Hq * d].unflatten(1, (Hq, d))
    s["k"] = rows[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
    s["q_out"] = torch.empty((n, Hq, d), dtype=dt, device="cuda")
    s["k_out"] = torch.empty((n, Hk, d), dtype=dt, device="cuda")
    if case["given"]:                       # (a block's rows: the depth in the draft)
        b = np.repeat(np.arange(case["B"]), new)
        at = np.arange(n) - np.repeat(np.cumsum(new) - new, new)
        s["positions"] = _cuda((held[b] + rs.integers(0, at + 1)).astype(np.int32))
    s["freqs"] = _cuda(_freqs(case))
    s["attention"] = ATTENTION if case["scaling"] == "ramp" else 1.0
    if own:
        bn = _package()
        s["desc"] = bn.rope_desc(n, Hq, Hk, d, case["rot"],
                                 bn.SPEC_ROPE_PAIRS if case["layout"] == "pairs" else bn.SPEC_ROPE_HALVES,
                                 bn.spec_dtype(s["q"]), s["attention"])
        kind = {"plain": bn.SPEC_ROPE_PLAIN, "linear": bn.SPEC_ROPE_LINEAR, "ramp": bn.SPEC_ROPE_RAMP}
        s["plan"] = bn.spec_rope_freqs(case["rot"], BASE, kind[case["scaling"]], FACTOR, TRAINED, LOW, HIGH)


# ---------------------------------------------------------------- one pass each

def run(s):
    return {"chunk": _run_chunk, "chunk8": _run_chunk, "append": _run_append,
            "rope": _run_rope}[s["op"]](s)


def _run_chunk(s):
    if own:
        bn = _package()
        call = bn.spec_chunk_attn_kv8 if s["op"] == "chunk8" else bn.spec_chunk_attn
        call(s["desc"], s["q"], s["cache"], s["seq_len"], s["cu_new"], s["o"], s["lse"], s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    Hq, Hkv, d, ps = (s["case"][k] for k in ("Hq", "Hkv", "d", "ps"))
    G, first = Hq // Hkv, 0
    for b, (n, S) in enumerate(zip(s["new"], s["held"])):      # (requests share no key)
        if n == 0:
            continue
        L = S + n
        if s["op"] == "chunk8":
            ids = s["page_table"][b, :-(-L // ps)].long()
            x = s["kv"].view(torch.uint8)[ids].view(F8).float() * s["scales"][ids].view(-1, Hkv, 1, 2, 1, 1)
            k, v = x.permute(3, 1, 0, 2, 4, 5).reshape(2, Hkv, -1, d)[:, :, :L]
        elif ps:
            ids = s["page_table"][b, :-(-L // ps)].long()
            k, v = (s[t][ids].permute(1, 0, 3, 2, 4).reshape(Hkv, -1, d)[:, :L].float() for t in "kv")
        else:
            k, v = s["k"][b, :, :L].float(), s["v"][b, :, :L].float()
        q = s["q"][first:first + n].float().view(n, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, G * n, d)
        t = torch.bmm(q, k.transpose(1, 2)).mul_(1 / math.sqrt(d)).view(Hkv, G, n, L)
        at = torch.arange(L, device="cuda")
        t.masked_fill_(at > at[S:, None], -math.inf)
        m = t.amax(-1, keepdim=True)
        p = t.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.bmm(p.view(Hkv, G * n, L), v).view(Hkv, G, n, d) / l
        s["o"][first:first + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, d).to(s["o"].dtype)
        s["lse"][first:first + n] = (m + l.log())[..., 0].permute(2, 0, 1).reshape(n, Hq)
        first += n
    return {"o": s["o"], "lse": s["lse"]}


def _run_append(s):
    if own:
        _package().kv_append(s["cache"], s["k"], s["v"], s["slot_map"])
    else:
        ps, d, slot = s["case"]["ps"], s["case"]["d"], s["slot_map"]
        rows = ps or s["k_cache"].shape[2]
        page, off = slot // rows, slot % rows
        for to, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
            if ps:
                to[page, :, :, off] = x.unflatten(2, (d // 64, 64))
            else:
                to[page, :, off] = x
    return {"k": s["k_cache"], "v": s["v_cache"]}


def _run_rope(s):
    c = s["case"]
    if own:
        where = dict(positions=s["positions"]) if c["given"] else dict(seq_len=s["seq_len"], cu_new=s["cu_new"])
        _package().spec_rope(s["desc"], s["plan"], s["q"], s["q_out"], s["k"], s["k_out"], **where)
        return {"q": s["q_out"], "k": s["k_out"]}
    r = c["rot"]
    if c["given"]:
        pos = s["positions"]
    else:
        i = torch.arange(s["q"].shape[0], device="cuda")
        b = torch.searchsorted(s["cu_new"][1:], i, right=True)
        pos = s["seq_len"][b] + i - s["cu_new"][b]
    a = pos.double()[:, None] * s["freqs"]
    cos, sin = (f(a).mul_(s["attention"]).float()[:, None] for f in (torch.cos, torch.sin))
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        y = x[..., :r].float()
        if c["layout"] == "pairs":
            u, w = y[..., 0::2], y[..., 1::2]
            z = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
        else:
            u, w = y[..., :r // 2], y[..., r // 2:]
            z = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
        out[..., :r] = z.to(out.dtype)
        out[..., r:] = x[..., r:]
    return {"q": s["q_out"], "k": s["k_out"]}


# --------------------------------------------------------------- what it takes

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    new, held = (x.astype(np.float64) for x in _new_and_held(case))
    n = new.sum()
    if case["op"] in ("chunk", "chunk8"):
        Hq, Hkv, d, ps = (case[k] for k in ("Hq", "Hkv", "d", "ps"))
        T = ((held + new) * (new > 0)).sum()                    # tokens that some query sees
        seen = (new * held + new * (new + 1) / 2).sum()
        by = n * Hq * (2 * d * e + 4) + 8 * case["B"]
        by += T * Hkv * 2 * d * (1 if case["op"] == "chunk8" else e)
        by += T * (4 + (8 * Hkv if case["op"] == "chunk8" else 0)) / ps if ps else 0
        return {"bytes": float(by), "flops": float(4 * d * Hq * seen)}
    if case["op"] == "append":
        by = n * (4 * case["Hkv"] * case["d"] * e + 8)
        return {"bytes": float(by), "flops": float(n * 2 * case["Hkv"] * case["d"])}
    heads = case["Hq"] + case["Hk"]
    by = n * (2 * heads * case["d"] * e + (4 if case["given"] else 0)) + 8 * case["B"]
    return {"bytes": float(by), "flops": float(n * 3 * heads * case["rot"])}


# ------------------------------------------------------- the definition in fp64

def exact(case, seed):
    if case["op"] == "append":              # (nothing is computed)
        return None
    if case["op"] == "rope":
        return _exact_rope(prepare(case, seed))
    return _exact_chunk(prepare(case, seed)) if work(case)["flops"] < 8e12 else None


def _exact_chunk(s):
    c = s["case"]
    Hq, Hkv, d, ps = (c[k] for k in ("Hq", "Hkv", "d", "ps"))
    G = Hq // Hkv
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    cu = s["cu_new"].cpu().numpy()
    for b in range(c["B"]):
        lo, hi, S = int(cu[b]), int(cu[b + 1]), int(s["seq_len"][b])
        if lo == hi:
            continue
        L = S + hi - lo
        t = torch.arange(L, device="cuda")
        if ps:
            page, off = s["page_table"][b].long()[t // ps], t % ps
        hidden = t[None, :] >= (S + 1 + torch.arange(hi - lo, device="cuda"))[:, None]
        for h in range(Hkv):
            if c["op"] == "chunk8":
                rows = [s["kv"].view(torch.uint8)[page, h, off // 8, x, off % 8].view(F8).double()
                        * s["scales"][page, h, x].double()[:, None] for x in (0, 1)]
            elif ps:
                rows = [s[x][page, h, :, off].double().reshape(L, d) for x in "kv"]
            else:
                rows = [s[x][b, h, :L].double() for x in "kv"]
            for hq in range(h * G, (h + 1) * G):
                w = (s["q"][lo:hi, hq].double() @ rows[0].T) / math.sqrt(d)
                w.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(w, 1)
                o[lo:hi, hq] = torch.exp_(w.sub_(z[:, None])) @ rows[1]
                lse[lo:hi, hq] = z
    return {"o": o, "lse": lse}


def _exact_rope(s):
    """On the host, a complex number a pair."""
    c = s["case"]
    r, out = c["rot"], {}
    if c["given"]:
        pos = s["positions"].cpu().numpy()
    else:
        pos = np.concatenate([S + np.arange(n) for n, S in zip(s["new"], s["held"])])
    turn = s["attention"] * np.exp(1j * pos[:, None, None].astype(np.float64) * _freqs(c))
    for name in ("q", "k"):
        x = s[name].double().cpu().numpy().copy()
        i = np.arange(0, r, 2) if c["layout"] == "pairs" else np.arange(r // 2)
        j = i + 1 if c["layout"] == "pairs" else i + r // 2
        z = (x[..., i] + 1j * x[..., j]) * turn
        x[..., i], x[..., j] = z.real, z.imag
        out[name] = torch.from_numpy(x)
    return out
