"""Cases of the 8-bit KV cache and logits operators: attention over the cache,
its two writers, the page planner and the logits adjustment.

``own`` False computes each operator in elementary torch operations; ``own``
True makes the library's calls on the same state.  An 8-bit cache holds, per
(page, KV head), one float8 e4m3 tile ``[page_size / 8][2][8][head_dim]`` (K
and V rows in alternating groups of eight) and one fp32 scale for K and one
for V; an element stands for code * scale.
"""

import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
E_MIN, E_MAX = -60, 60        # exponents that the writers give a scale


def _package():
    from self_speculative_verification_gb300 import binding
    return binding


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # attention: the smallest call (fp32, a lookahead block of four rows)
        dict(name="attn_tiny_f32", op="attn", B=2, Hq=4, Hkv=2, d=64, R=4, mask="la", soft=0,
             lo=128, hi=200, ps=16, dtype="f32"),
        # one token per request: plain decoding over the same cache
        dict(name="attn_decode", op="attn", B=16, Hq=32, Hkv=8, d=128, R=1, mask="chain", soft=0,
             lo=512, hi=4096, ps=16, dtype="bf16"),
        # a draft tree with contemplate rows and a soft prompt: many rows per head
        dict(name="attn_tree", op="attn", B=8, Hq=32, Hkv=8, d=128, R=120, mask="tree", soft=16,
             lo=256, hi=2048, ps=16, dtype="bf16"),
        # long contexts, a lookahead block of eight rows: the whole cache is read once
        dict(name="attn_long", op="attn", B=64, Hq=32, Hkv=8, d=128, R=8, mask="la", soft=0,
             lo=16384, hi=32768, ps=16, dtype="bf16"),
        # the accepted rows of a verification step enter the cache
        dict(name="commit_heads32", op="commit", B=16, Hkv=32, d=128, R=8, cap=8, lo=200, hi=600,
             ps=16, dtype="bf16"),
        # the same for long deep trees, fp32 keys, wider pages
        dict(name="commit_tree_f32", op="commit", B=64, Hkv=8, d=128, R=64, cap=24, lo=100, hi=900,
             ps=32, dtype="f32"),
        # one chunk of a few prompts enters the cache
        dict(name="append_chunk", op="append", B=5, Hkv=8, d=128, lo=1, hi=120, held=70, ps=16,
             dtype="bf16", pad=0),
        # whole prompts, rows a part of wider projection rows
        dict(name="append_prompts", op="append", B=32, Hkv=8, d=128, lo=100, hi=2048, held=0, ps=16,
             dtype="bf16", pad=4096),
        # pages and slots of one decoding step
        dict(name="plan_step", op="plan", B=64, lo=1, hi=8, held=30000, ps=16),
        # pages and slots of a batch of prompts
        dict(name="plan_prompts", op="plan", B=200, lo=1, hi=4096, held=5000, ps=16),
        # penalties, biases and grammar masks ahead of a lookahead acceptance
        dict(name="logits_la", op="logits", B=16, Rj=8, V=32000, hist=4096, N=8, n_bias=32,
             n_masks=4, dtype="bf16"),
        # the same on every node of a draft tree over a large vocabulary
        dict(name="logits_tree", op="logits", B=8, Rj=60, V=128256, hist=2048, N=60, n_bias=64,
             n_masks=8, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "commit", "append", "plan", "logits"])
    if op == "attn":
        dtype = rng.choice(["bf16"] * 7 + ["f32"])
        d = rng.choice([64, 128, 128, 128])
        Hkv = rng.choice([1, 2, 4, 8, 16, 32])
        G = rng.choice([1, 1, 2, 4, 7, 8])
        mask = rng.choice(["la", "chain", "tree"])
        R = rng.choice([1, 1, _log(rng, 1, 16), _log(rng, 2, 160)])
        hi = _log(rng, 8, 32768)
        B = max(1, min(_log(rng, 1, 64), int(4e8 / (hi * Hkv * d))))
        if dtype == "f32" or R * G > 64:       # (bounded by arithmetic, not by the bytes)
            B = max(1, min(B, int(6e9 / (hi * Hkv * d * R * G))))
            hi = min(hi, max(8, int(6e9 / (B * Hkv * d * R * G))))
        return dict(op=op, B=B, Hq=Hkv * G, Hkv=Hkv, d=d, R=R, mask=mask,
                    soft=rng.choice([0, 0, rng.randint(1, 64)]), lo=rng.choice([0, 1, hi // 2, hi]),
                    hi=hi, ps=rng.choice([16, 16, 32, 48, 64, 128]), dtype=dtype)
    if op == "commit":
        R = _log(rng, 1, 128)
        hi = _log(rng, 16, 1500)
        Hkv = rng.choice([1, 4, 8, 32])
        return dict(op=op, B=max(1, min(_log(rng, 1, 100), int(6e5 / (hi * Hkv)))), Hkv=Hkv,
                    d=rng.choice([64, 128]), R=R, cap=rng.randint(1, max(1, min(R, 40))),
                    lo=rng.randint(1, hi), hi=hi, ps=rng.choice([16, 32, 48, 64]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "append":
        hi = _log(rng, 2, 4096)
        Hkv = rng.choice([1, 4, 8, 32])
        return dict(op=op, B=max(1, min(_log(rng, 1, 64), int(2e5 / (hi * Hkv)))), Hkv=Hkv,
                    d=rng.choice([64, 128]), lo=rng.randint(0, hi // 2), hi=hi,
                    held=rng.choice([0, rng.randint(1, 300)]), ps=rng.choice([16, 32, 64, 128]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 64, 1024]))
    if op == "plan":
        hi = _log(rng, 1, 4096)
        return dict(op=op, B=max(1, min(_log(rng, 1, 2000), int(1.6e6 / hi))), lo=rng.randint(0, hi),
                    hi=hi, held=_log(rng, 1, 30000), ps=rng.choice([16, 32, 48, 64, 128]))
    V = _log(rng, 500, 130000)
    rows = max(1, min(_log(rng, 1, 512), int(6e7 / V)))
    Rj = rng.choice([1, _log(rng, 1, 64)])
    Rj = min(Rj, rows)
    return dict(op="logits", B=max(1, rows // Rj), Rj=Rj, V=V, hist=_log(rng, 1, 16384), N=max(Rj, 2),
                n_bias=rng.choice([0, _log(rng, 1, 300)]), n_masks=rng.choice([0, 1, 5]),
                dtype=rng.choice(["bf16", "bf16", "f32"]))


# ------------------------------------------------------------------- the states

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62) + 17)


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _lengths(rs, case, held=None):
    """Lengths in [lo, hi] (with `held`, also what each request holds before):
    a case has the same ones under every seed, in another order."""
    fixed = np.random.default_rng([case["lo"], case["hi"], case["B"]])
    n = fixed.integers(case["lo"], case["hi"] + 1, size=case["B"])
    n[0] = case["hi"]
    order = rs.permutation(case["B"])
    if held is None:
        return n[order]
    return n[order], fixed.integers(0, held + 1, size=case["B"])[order]


def _pages(rs, held, room, ps):
    """Page tables for requests that hold `held` tokens and may come to hold
    `room`: (n_pages, table int32 [B][max_pages], the free pages in list order)."""
    need, cap = -(-held // ps), max(1, int((-(-room // ps)).max()))
    spare = int((-(-room // ps) - need).sum()) + 4
    n_pages = int(need.sum()) + spare
    perm = rs.permutation(n_pages).astype(np.int32)
    table = np.zeros((len(held), cap), dtype=np.int32)
    cols = np.arange(cap)[None, :]
    mine = cols < need[:, None]
    table[mine] = perm[:int(need.sum())]
    return n_pages, table, perm[int(need.sum()):]


def _filled_cache(g, n_pages, Hkv, ps, d):
    """A cache whose every block holds normal keys and values of its own
    size (heads and pages differ in size, as they do in a trained model)."""
    kv = torch.empty((n_pages, Hkv, ps // 8, 2, 8, d), dtype=F8, device="cuda")
    scales = torch.empty((n_pages, Hkv, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 27) // (Hkv * ps * 2 * d))
    head = torch.exp2(torch.randint(-2, 2, (1, Hkv, 1), generator=g, device="cuda").float())
    head = head.expand(1, Hkv, 2).clone()
    head[:, :, 0] = 1.0
    for lo in range(0, n_pages, step):
        n = min(step, n_pages - lo)
        x = torch.randn((n, Hkv, ps // 8, 2, 8, d), generator=g, device="cuda")
        x = x * head.view(1, Hkv, 1, 2, 1, 1)
        a = x.abs().amax(dim=(2, 4, 5))
        e = _exponent(a)
        s = torch.ldexp(torch.ones_like(a), e)
        scales[lo:lo + n] = s
        kv[lo:lo + n] = (x / s.view(n, Hkv, 1, 2, 1, 1)).to(F8)
    return kv, scales


def _exponent(a):
    """The smallest e with a <= 448 * 2^e, within [E_MIN, E_MAX]."""
    m, x = torch.frexp(a)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX).to(torch.int32)


def _parents(rs, case):
    """Parent row of every block row (-1: none, -2: padding), and which rows
    see the soft prompt."""
    B, R = case["B"], case["R"]
    par = np.full((B, R), -1, dtype=np.int64)
    soft = np.zeros((B, R), dtype=bool)
    if case["mask"] == "chain":
        par[:] = np.arange(R) - 1
    elif case["mask"] == "tree":
        for r in range(1, R):
            par[:, r] = rs.integers(max(0, r - 9), r, size=B)
        soft[:, R // 2:] = True
    if R > 2:
        pad = rs.integers(0, max(1, R // 4), size=B)
        par[np.arange(R)[None, :] >= (R - pad)[:, None]] = -2
        soft &= par != -2
    return par, soft


def prepare(case, seed):
    g, rs = _gen(seed), np.random.default_rng([seed, 5])
    return {"attn": _prepare_attn, "commit": _prepare_commit, "append": _prepare_append,
            "plan": _prepare_plan, "logits": _prepare_logits}[case["op"]](case, g, rs)


def _cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _randn(g, shape, dt):
    return torch.randn(shape, generator=g, device="cuda").to(dt)


def _prepare_attn(case, g, rs):
    B, Hq, Hkv, d, R, ps, ns = (case[k] for k in ("B", "Hq", "Hkv", "d", "R", "ps", "soft"))
    dt = _dt(case)
    S = _lengths(rs, case)
    n_pages, table, _ = _pages(rs, S, S, ps)
    kv, scales = _filled_cache(g, n_pages, Hkv, ps, d)
    par, soft = _parents(rs, case)
    vis = np.zeros((B, R, R), dtype=bool)
    for r in range(R):
        up = par[:, r] >= 0
        vis[up, r] = vis[np.nonzero(up)[0], par[up, r]]
        vis[par[:, r] != -2, r, r] = True
    W = (R + 31) // 32
    bits = np.zeros((B, R, W * 32), dtype=np.uint8)
    bits[:, :, :R] = vis
    words = np.packbits(bits, axis=2, bitorder="little").view(np.int32)
    flags = ((par != -2) * 1 + soft * 2).astype(np.uint8)
    s = dict(op="attn", case=dict(case), seq_len=_cuda(S.astype(np.int32)), longest=int(S.max()),
             kv=kv, scales=scales, page_table=_cuda(table), q=_randn(g, (B, R, Hq, d), dt),
             kb=_randn(g, (B, Hkv, R, d), dt), vb=_randn(g, (B, Hkv, R, d), dt),
             soft_k=_randn(g, (Hkv, ns, d), dt) if ns else None,
             soft_v=_randn(g, (Hkv, ns, d), dt) if ns else None,
             vis=_cuda(words.reshape(B, R, W)), row_flags=_cuda(flags),
             o=torch.empty((B, R, Hq, d), dtype=dt, device="cuda"),
             lse=torch.empty((B, Hq, R), dtype=torch.float32, device="cuda"))
    if own:
        bn = _package()
        s["cache"] = bn.kv8_desc(s["kv"], s["scales"], s["page_table"])
        s["attn"] = bn.attn_desc(B, R, Hq, Hkv, d, bn.spec_dtype(s["q"]), ns)
        n = bn.spec_verify_attn_kv8_workspace_size(s["attn"], s["cache"])
        s["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    return s


def _row_sizes(g, shape):
    """Sizes of new rows: now and then one that outgrows its block's scale."""
    u = torch.rand(shape, generator=g, device="cuda")
    return torch.exp2(torch.floor(u * 3 - 1)) * torch.where(u > 0.95, 8.0, 1.0)


def _prepare_commit(case, g, rs):
    B, Hkv, d, R, cap, ps = (case[k] for k in ("B", "Hkv", "d", "R", "cap", "ps"))
    dt = _dt(case)
    S = np.maximum(1, _lengths(rs, case))
    acc = rs.integers(0, cap + 1, size=B)
    path = np.full((B, cap), -1, dtype=np.int32)
    for b in range(B):
        path[b, :acc[b]] = np.sort(rs.choice(R, size=acc[b], replace=False))
    n_pages, table, free = _pages(rs, S, S + cap, ps)
    kv, scales = _filled_cache(g, n_pages, Hkv, ps, d)
    size = _row_sizes(g, (B, Hkv, R, 1))
    s = dict(op="commit", case=dict(case), kv=kv, scales=scales, page_table=_cuda(table),
             kb=(_randn(g, (B, Hkv, R, d), torch.float32) * size).to(dt),
             vb=(_randn(g, (B, Hkv, R, d), torch.float32) * size).to(dt), path=_cuda(path),
             acc_len=_cuda(acc.astype(np.int32)), seq_len0=_cuda(S.astype(np.int32)),
             seq_len=_cuda(S.astype(np.int32)), free_pages=_cuda(free),
             free_head=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if own:
        s["cache"] = _package().kv8_desc(s["kv"], s["scales"], s["page_table"])
    return s


def _slots(table, held, new, ps):
    """Slot of every new token of the packed batch (page * page_size + offset)."""
    b = np.repeat(np.arange(len(new)), new)
    pos = held[b] + np.arange(new.sum()) - np.repeat(np.cumsum(new) - new, new)
    return table[b, pos // ps].astype(np.int64) * ps + pos % ps


def _prepare_append(case, g, rs):
    B, Hkv, d, ps = (case[k] for k in ("B", "Hkv", "d", "ps"))
    dt = _dt(case)
    new, held = _lengths(rs, case, case["held"])
    n_pages, table, _ = _pages(rs, held + new, held + new, ps)
    kv, scales = _filled_cache(g, n_pages, Hkv, ps, d)
    n, width = int(new.sum()), 2 * Hkv * d + case["pad"]
    rows = (torch.randn((n, width), generator=g, device="cuda")
            * _row_sizes(g, (n, 1))).to(dt)
    return dict(op="append", case=dict(case), kv=kv, scales=scales,
                slot_map=_cuda(_slots(table, held, new, ps)), rows=rows,
                k=rows[:, :Hkv * d].unflatten(1, (Hkv, d)),
                v=rows[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d)),
                **({"cache": _package().kv8_desc(kv, scales)} if own else {}))


def _prepare_plan(case, g, rs):
    B, ps = case["B"], case["ps"]
    new, held = _lengths(rs, case, case["held"])
    n_pages, table, free = _pages(rs, held, held + new, ps)
    i32 = dict(dtype=torch.int32, device="cuda")
    n_slots = int(new.sum()) + 13          # (a buffer for batches up to a size)
    return dict(op="plan", case=dict(case), seq_len=_cuda(held.astype(np.int32)),
                n_new=_cuda(new.astype(np.int32)), n_pages=n_pages, page_table=_cuda(table),
                free_pages=_cuda(free), free_head=torch.zeros(1, **i32),
                cu_new=torch.zeros(B + 1, **i32), new_len=torch.zeros(B, **i32),
                slot_map=torch.zeros(n_slots, dtype=torch.int64, device="cuda"))


def _prepare_logits(case, g, rs):
    B, Rj, V, N, nb = (case[k] for k in ("B", "Rj", "V", "N", "n_bias"))
    dt = _dt(case)
    hl = rs.integers(0, case["hist"] + 1, size=B)
    hl[rs.integers(0, B)] = case["hist"]
    # tokens come again as they do in text: a few are frequent
    hist = np.minimum(V - 1, (V * rs.random((B, case["hist"])) ** 4)).astype(np.int32)
    tokens = np.minimum(V - 1, (V * rs.random((B, N)) ** 4)).astype(np.int32)
    parent = np.full((B, N), -1, dtype=np.int32)
    for c in range(1, N):
        parent[:, c] = rs.integers(max(0, c - 6), c, size=B)
    s = dict(op="logits", case=dict(case), logits=_randn(g, (B, Rj, V), torch.float32).mul_(3).to(dt),
             history=_cuda(hist), hist_len=_cuda(hl.astype(np.int32)),
             n_prompt=_cuda((hl * rs.random(B)).astype(np.int32)), tokens=_cuda(tokens),
             tree_parent=_cuda(parent),
             row_node=_cuda(rs.integers(-1, N, size=(B, Rj)).astype(np.int32)),
             repetition=_cuda(rs.uniform(0.9, 1.4, size=B).astype(np.float32)),
             presence=_cuda(rs.uniform(-0.2, 0.8, size=B).astype(np.float32)),
             frequency=_cuda(rs.uniform(0.0, 0.5, size=B).astype(np.float32)),
             bias_ids=None, bias=None, mask_bits=None, row_mask=None)
    if nb:
        ids = rs.integers(-1, V, size=(B, nb)).astype(np.int32)
        s["bias_ids"] = _cuda(ids)
        s["bias"] = _cuda(rs.normal(0, 3, size=(B, nb)).astype(np.float32))
    if case["n_masks"]:
        W = (V + 31) // 32
        words = rs.integers(0, 1 << 32, size=(case["n_masks"], W), dtype=np.uint32)
        words[0] &= rs.integers(0, 1 << 32, size=W, dtype=np.uint32)
        words[0] &= rs.integers(0, 1 << 32, size=W, dtype=np.uint32)
        s["mask_bits"] = _cuda(words.view(np.int32))
        s["row_mask"] = _cuda(rs.integers(-1, case["n_masks"], size=(B, Rj)).astype(np.int32))
    s["out"] = torch.empty_like(s["logits"])
    if own:
        bn = _package()
        s["desc"] = bn.logits_desc(B, Rj, V, bn.spec_dtype(s["logits"]), N, case["hist"], nb,
                                   case["n_masks"])
    return s


# ---------------------------------------------------------------- one pass each

def run(s):
    return {"attn": _run_attn, "commit": _run_commit, "append": _run_append, "plan": _run_plan,
            "logits": _run_logits}[s["op"]](s)


def _run_attn(s):
    if own:
        _package().spec_verify_attn_kv8(s["attn"], s["q"], s["cache"], s["kb"], s["vb"], s["soft_k"],
                                        s["soft_v"], s["seq_len"], s["vis"], s["row_flags"], s["o"],
                                        s["lse"], s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    B, Hq, Hkv, d, R, ps, ns = (s["case"][k] for k in ("B", "Hq", "Hkv", "d", "R", "ps", "soft"))
    G, n = Hq // Hkv, -(-s["longest"] // ps)
    pages = s["page_table"][:, :n].long()
    x = s["kv"].view(torch.uint8)[pages].view(F8).float()
    x = x * s["scales"][pages].view(B, n, Hkv, 1, 2, 1, 1)
    x = x.permute(4, 0, 2, 1, 3, 5, 6).reshape(2, B, Hkv, n * ps, d)
    own_kv = torch.stack([s["kb"].float(), s["vb"].float()])
    parts = [x]
    if ns:
        soft = torch.stack([s["soft_k"].float(), s["soft_v"].float()])
        parts.append(soft[:, None].expand(2, B, Hkv, ns, d))
    parts.append(own_kv)
    k, v = torch.cat(parts, 3)
    at = torch.arange(n * ps, device="cuda")
    valid = (s["row_flags"] & 1).bool()[:, :, None]
    bits = (s["vis"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    seen = [valid & (at < s["seq_len"][:, None])[:, None, :]]
    if ns:
        seen.append((valid & (s["row_flags"] & 2).bool()[:, :, None]).expand(B, R, ns))
    seen.append(valid & bits.reshape(B, R, -1)[:, :, :R].bool())
    seen = torch.cat(seen, 2)[:, None, :, None, :]
    q = s["q"].float().view(B, R, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, R * G, d)
    t = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(B, Hkv, R, G, -1)
    t = t.masked_fill_(~seen, -math.inf)
    m = t.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = t.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, R * G, -1) @ v
    o = torch.where(l > 0, o.view(B, Hkv, R, G, d) / l, torch.zeros((), device="cuda"))
    lse = (m + l.log())[..., 0].permute(0, 1, 3, 2).reshape(B, Hq, R)
    return {"o": o.permute(0, 2, 1, 3, 4).reshape(B, R, Hq, d).to(s["q"].dtype), "lse": lse}


def _merge(kv, scales, page, first, count, k, v, src, ps):
    """Writes new rows into blocks: block i takes rows src[i, t] (of k, v
    [rows][Hkv][d] after `src` indexing: [n, ps, Hkv, d]) at offsets first[i]
    .. first[i] + count[i] - 1.  A block whose first new row is its first row
    takes a scale of its own; otherwise the scale only grows, and the rows
    before the new ones are rounded to it again."""
    n, Hkv, d = page.numel(), kv.shape[1], kv.shape[5]
    at = torch.arange(ps, device="cuda")
    fresh = (first == 0) & (count > 0)
    new = (at >= first[:, None]) & (at < (first + count)[:, None])          # [n, ps]
    old = at < first[:, None]
    rows = torch.stack([k[src], v[src]], 2).float()                         # [n, ps, 2, Hkv, d]
    a = (rows.abs() * new[:, :, None, None, None]).amax((1, 4))             # [n, 2, Hkv]
    s_new = torch.ldexp(torch.ones_like(a), _exponent(a)).permute(0, 2, 1)  # [n, Hkv, 2]
    s_old = scales[page]
    s = torch.where(fresh[:, None, None], s_new, torch.maximum(s_old, s_new))
    s = torch.where((count > 0)[:, None, None], s, s_old)
    codes = kv.view(torch.uint8)[page].view(F8)
    was = codes.float().permute(0, 2, 4, 3, 1, 5).reshape(n, ps, 2, Hkv, d)
    r = (s_old / s).permute(0, 2, 1)[:, None, :, :, None]
    keep = torch.where(old[:, :, None, None, None], was * r, was)
    x = torch.where(new[:, :, None, None, None], rows / s.permute(0, 2, 1)[:, None, :, :, None],
                    keep).to(F8)
    x = x.view(torch.uint8).view(n, ps // 8, 8, 2, Hkv, d).permute(0, 4, 1, 3, 2, 5)
    kv.view(torch.uint8)[page] = x
    scales[page] = s


def _run_commit(s):
    s["seq_len"].copy_(s["seq_len0"])
    s["free_head"].zero_()
    if own:
        _package().kv8_commit(s["cache"], s["kb"], s["vb"], s["path"], s["acc_len"], s["seq_len"],
                              s["free_pages"], s["free_head"])
    else:
        B, Hkv, d, R, cap, ps = (s["case"][k] for k in ("B", "Hkv", "d", "R", "cap", "ps"))
        S, a, table = s["seq_len"].long(), s["acc_len"].long(), s["page_table"]
        had, want = -(-S // ps), -(-(S + a) // ps)
        start = torch.cumsum(want - had, 0) - (want - had)
        cols = torch.arange(table.shape[1], device="cuda")
        i = (start[:, None] + cols - had[:, None]).clamp(0, s["free_pages"].numel() - 1)
        takes = (cols >= had[:, None]) & (cols < want[:, None])
        table.copy_(torch.where(takes, s["free_pages"][i], table))
        # the blocks from the first new row's to the last one's (a request
        # with fewer, or none, names its last one again, with the same rows)
        J = -(-cap // ps) + 1
        j0 = torch.minimum(S // ps, want - 1)
        j = torch.minimum(j0[:, None] + torch.arange(J, device="cuda"), (want - 1)[:, None])
        page = torch.gather(table.long(), 1, j)
        first = (S[:, None] - j * ps).clamp(min=0)
        count = ((S + a)[:, None] - j * ps).clamp(max=ps) - first
        at = torch.arange(ps, device="cuda")
        nth = (j[:, :, None] * ps + at - S[:, None, None]).clamp(0, cap - 1)
        row = torch.gather(s["path"].long(), 1, nth.view(B, -1)).view(B, J, ps).clamp(min=0)
        src = row + (torch.arange(B, device="cuda") * R)[:, None, None]
        flat = lambda x: x.transpose(1, 2).reshape(B * R, Hkv, d)  # noqa: E731
        _merge(s["kv"], s["scales"], page.view(-1), first.view(-1), count.view(-1), flat(s["kb"]),
               flat(s["vb"]), src.view(B * J, ps), ps)
        s["seq_len"].add_(s["acc_len"])
        s["free_head"].add_((want - had).sum().to(torch.int32))
    return {k: s[k] for k in ("kv", "scales", "page_table", "seq_len", "free_head")}


def _run_append(s):
    if own:
        _package().kv8_append(s["cache"], s["k"], s["v"], s["slot_map"])
    else:
        ps, slot = s["case"]["ps"], s["slot_map"]
        n = slot.numel()
        i = torch.arange(n, device="cuda")
        page, off = slot // ps, slot % ps
        # every token names the run of tokens that shares its page
        head = torch.ones(n, dtype=torch.bool, device="cuda")
        head[1:] = (page[1:] != page[:-1])
        start = torch.cummax(torch.where(head, i, torch.zeros_like(i)), 0).values
        starts = torch.unique_consecutive(start)
        ends = torch.cat([starts[1:], torch.full_like(starts[:1], n)])
        at = torch.arange(ps, device="cuda")
        first = off[starts]
        src = (starts[:, None] + at - first[:, None]).clamp(0, n - 1)
        _merge(s["kv"], s["scales"], page[starts], first, ends - starts, s["k"], s["v"], src, ps)
    return {"kv": s["kv"], "scales": s["scales"]}


def _run_plan(s):
    s["free_head"].zero_()
    if own:
        _package().spec_page_plan(s["case"]["ps"], s["n_pages"], s["seq_len"], s["n_new"],
                                  s["page_table"], s["free_pages"], s["free_head"], s["cu_new"],
                                  s["slot_map"], s["new_len"])
    else:
        ps, table = s["case"]["ps"], s["page_table"]
        S, a = s["seq_len"].long(), s["n_new"].long()
        had, want = -(-S // ps), -(-(S + a) // ps)
        start = torch.cumsum(want - had, 0) - (want - had)
        cols = torch.arange(table.shape[1], device="cuda")
        i = (start[:, None] + cols - had[:, None]).clamp(0, s["free_pages"].numel() - 1)
        takes = (cols >= had[:, None]) & (cols < want[:, None])
        table.copy_(torch.where(takes, s["free_pages"][i], table))
        s["free_head"].add_((want - had).sum().to(torch.int32))
        cu = torch.cumsum(a, 0)
        s["cu_new"][1:] = cu
        s["new_len"].copy_(S + a)
        t = torch.arange(s["slot_map"].numel(), device="cuda")
        b = torch.searchsorted(cu, t, right=True).clamp(max=S.numel() - 1)
        pos = (S[b] + t - (cu - a)[b]).clamp(max=table.shape[1] * ps - 1)
        slot = table[b, pos // ps].long() * ps + pos % ps
        s["slot_map"].copy_(torch.where(t < cu[-1], slot, torch.full_like(slot, -1)))
    return {k: s[k] for k in ("page_table", "free_head", "cu_new", "slot_map", "new_len")}


def _run_logits(s):
    if own:
        _package().spec_logits_adjust(s["desc"], s["logits"], s["out"], s["history"], s["hist_len"],
                                      s["n_prompt"], s["tokens"], s["tree_parent"], s["row_node"],
                                      s["repetition"], s["presence"], s["frequency"], s["bias_ids"],
                                      s["bias"], s["mask_bits"], s["row_mask"])
        return {"out": s["out"]}
    B, Rj, V, N = (s["case"][k] for k in ("B", "Rj", "V", "N"))
    at = torch.arange(s["history"].shape[1], device="cuda")
    held = at < s["hist_len"][:, None]
    said = held & (at >= s["n_prompt"][:, None])
    zero = torch.zeros((B, V), device="cuda")
    ids = s["history"].long()
    count = zero.scatter_add(1, ids, said.float())
    prompt = zero.scatter_add(1, ids, held.float())
    # nodes on the path to each row's node: the closure of the parents
    up = torch.zeros((B, N + 1, N + 1), device="cuda")
    up.scatter_(2, torch.arange(N + 1, device="cuda")[None, :, None].expand(B, N + 1, 1), 1.0)
    par = torch.cat([torch.zeros_like(s["tree_parent"][:, :1]), s["tree_parent"] + 1], 1).long()
    up.scatter_(2, par[:, :, None], 1.0)
    steps = max(1, math.ceil(math.log2(N + 1)))
    up = (torch.matrix_power(up, 1 << steps) > 0).float()
    path = torch.gather(up, 1, (s["row_node"] + 1).long()[:, :, None].expand(B, Rj, N + 1))[:, :, 1:]
    z = s["logits"].float()
    more = torch.zeros_like(z).scatter_add_(2, s["tokens"].long()[:, None].expand(B, Rj, N), path)
    n = more.add_(count[:, None])
    seen = (n > 0) | (prompt > 0)[:, None]
    rep = s["repetition"][:, None, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None, None] * n - s["presence"][:, None, None] * (n > 0)
    if s["bias_ids"] is not None:
        on = s["bias_ids"] >= 0
        z = z + zero.scatter_add(1, s["bias_ids"].clamp(min=0).long(), s["bias"] * on)[:, None]
    if s["mask_bits"] is not None:
        bits = (s["mask_bits"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
        allowed = bits.reshape(bits.shape[0], -1)[:, :V].bool()[s["row_mask"].clamp(min=0).long()]
        z = torch.where(allowed | (s["row_mask"] < 0)[..., None], z, torch.full_like(z, -math.inf))
    return {"out": z.to(s["logits"].dtype)}


# --------------------------------------------------------------- what it takes

def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    op = case["op"]
    if op == "attn":
        B, Hq, Hkv, d, R, ps, ns = (case[k] for k in ("B", "Hq", "Hkv", "d", "R", "ps", "soft"))
        T = B * (case["lo"] + case["hi"]) / 2
        by = T * Hkv * (2 * d + 8 / ps) + 4 * T / ps                     # codes, scales, page table
        by += B * R * (2 * Hq * d * e + 2 * Hkv * d * e + 4 * Hq + 4 * ((R + 31) // 32) + 1)
        by += ns * Hkv * 2 * d * e
        return {"bytes": by, "flops": 4 * d * Hq * R * (T + B * (ns + min(R, 8)))}
    if op == "commit":
        rows = case["B"] * case["cap"] / 2
        # the new rows in and out, and each block's scales
        by = rows * case["Hkv"] * 2 * case["d"] * (e + 1) + case["B"] * case["Hkv"] * 16
        return {"bytes": by, "flops": rows * case["Hkv"] * 2 * case["d"] * 2}
    if op == "append":
        rows = case["B"] * (case["lo"] + case["hi"]) / 2
        by = rows * case["Hkv"] * (2 * case["d"] * (e + 1) + 8 / case["ps"]) + 8 * rows
        return {"bytes": by, "flops": rows * case["Hkv"] * 2 * case["d"] * 2}
    if op == "plan":
        rows = case["B"] * (case["lo"] + case["hi"]) / 2
        return {"bytes": 8 * rows + 8 * rows / case["ps"] + 20 * case["B"], "flops": 2 * rows}
    n = case["B"] * case["Rj"] * case["V"]
    by = 2 * e * n + 4 * case["B"] * (case["hist"] / 2 + 2 * case["N"] + 2 * case["n_bias"])
    by += case["n_masks"] * case["V"] / 8
    return {"bytes": by, "flops": 4 * n}


# ------------------------------------------------------- the definition in fp64

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "commit": _exact_commit, "append": _exact_append,
            "plan": lambda s: None, "logits": _exact_logits}[case["op"]](s)


def _exact_attn(s):
    c = s["case"]
    B, Hq, Hkv, d, R, ps = (c[k] for k in ("B", "Hq", "Hkv", "d", "R", "ps"))
    o = torch.zeros((B, R, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, R), -math.inf, dtype=torch.float64, device="cuda")
    table, words = s["page_table"].cpu().numpy(), s["vis"].cpu().numpy().view(np.uint32)
    flags, lens = s["row_flags"].cpu().numpy(), s["seq_len"].cpu().numpy()
    for b in range(B):
        S = int(lens[b])
        ids = torch.from_numpy(table[b, :-(-S // ps)].astype(np.int64)).cuda()
        blk = s["kv"].view(torch.uint8).index_select(0, ids).view(F8).double()
        sc = s["scales"].index_select(0, ids).double()
        see = np.unpackbits(words[b].view(np.uint8), axis=1, bitorder="little")[:, :R].astype(bool)
        for h in range(Hkv):
            kv = []
            for x, sk, sb in ((0, "soft_k", "kb"), (1, "soft_v", "vb")):
                t = blk[:, h, :, x].reshape(-1, ps, d) * sc[:, h, x].view(-1, 1, 1)
                t = [t.reshape(-1, d)[:S]] + ([s[sk][h].double()] if c["soft"] else [])
                kv.append(torch.cat(t + [s[sb][b, h].double()]))
            q = s["q"][b, :, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
            w = torch.einsum("rgd,td->grt", q, kv[0]) / math.sqrt(d)
            mask = np.concatenate([np.ones((R, S), bool),
                                   np.repeat((flags[b] & 2)[:, None] != 0, c["soft"], 1), see], 1)
            mask &= (flags[b] & 1)[:, None] != 0
            w.masked_fill_(torch.from_numpy(~mask).cuda(), -math.inf)
            z = torch.logsumexp(w, 2)
            p = torch.exp(w - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            o[b, :, hs] = torch.einsum("grt,td->rgd", p, kv[1])
            lse[b, hs] = z
    return {"o": o, "lse": lse}


def _round_e4m3(x):
    """Nearest e4m3 value (ties to even), |x| <= 448, in float64."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -30)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.round(x / step) * step


class _Blocks:
    """A host copy of a cache as values in float64, written a run of rows at a time."""

    def __init__(self, s):
        x = s["kv"].double().cpu().numpy()                    # codes
        n, H, g, _, _, d = x.shape
        self.codes = x.transpose(0, 3, 2, 4, 1, 5).reshape(n, 2, g * 8, H, d).copy()
        self.scales = s["scales"].double().cpu().numpy().copy()

    def put(self, page, off, rows):
        """rows [2][n][Hkv][d] at offsets off.. of one page."""
        n = rows.shape[1]
        a = np.abs(rows).max((1, 3))                          # [2][Hkv]
        e = np.ceil(np.log2(np.maximum(a, 2.0 ** -100) / 448.0))
        need = 2.0 ** np.clip(e, E_MIN, E_MAX)
        was = self.scales[page].T                             # [2][Hkv]
        s = need if off == 0 else np.maximum(was, need)
        if off:
            r = (was / s)[:, None, :, None]
            self.codes[page][:, :off] = _round_e4m3(self.codes[page][:, :off] * r)
        self.codes[page][:, off:off + n] = _round_e4m3(rows / s[:, None, :, None])
        self.scales[page] = s.T

    def out(self):
        n, _, ps, H, d = self.codes.shape
        x = self.codes.reshape(n, 2, ps // 8, 8, H, d).transpose(0, 4, 2, 1, 3, 5)
        return torch.from_numpy(np.ascontiguousarray(x)), torch.from_numpy(self.scales)


def _exact_commit(s):
    if s["kv"].numel() > 3e8:
        return None
    ps, blocks = s["case"]["ps"], _Blocks(s)
    table, free = s["page_table"].cpu().numpy().copy(), list(s["free_pages"].cpu().numpy())
    k, v = s["kb"].double().cpu().numpy(), s["vb"].double().cpu().numpy()
    path, acc, lens = (s[n].cpu().numpy() for n in ("path", "acc_len", "seq_len0"))
    for b in range(len(acc)):
        done = 0
        while done < acc[b]:
            pos = int(lens[b]) + done
            if pos % ps == 0:
                table[b, pos // ps] = free.pop(0)
            n = min(ps - pos % ps, int(acc[b]) - done)
            r = path[b, done:done + n]
            rows = np.stack([k[b][:, r], v[b][:, r]]).transpose(0, 2, 1, 3)
            blocks.put(table[b, pos // ps], pos % ps, rows)
            done += n
    kv, scales = blocks.out()
    return {"kv": kv, "scales": scales, "page_table": None, "seq_len": None, "free_head": None}


def _exact_append(s):
    if s["kv"].numel() > 3e8:
        return None
    ps, blocks = s["case"]["ps"], _Blocks(s)
    slot = s["slot_map"].cpu().numpy()
    k, v = s["k"].double().cpu().numpy(), s["v"].double().cpu().numpy()
    i = 0
    while i < len(slot):
        page, off = divmod(int(slot[i]), ps)
        n = 1
        while i + n < len(slot) and off + n < ps and slot[i + n] == slot[i] + n:
            n += 1
        blocks.put(page, off, np.stack([k[i:i + n], v[i:i + n]]))
        i += n
    kv, scales = blocks.out()
    return {"kv": kv, "scales": scales}


def _exact_logits(s):
    c = s["case"]
    z = s["logits"].double().cpu().numpy()
    get = lambda n: None if s[n] is None else s[n].cpu().numpy()  # noqa: E731
    hist, hl, npm, tok, par, node = map(get, ("history", "hist_len", "n_prompt", "tokens",
                                              "tree_parent", "row_node"))
    rep, pres, freq, ids, bias, bits, row_mask = map(get, (
        "repetition", "presence", "frequency", "bias_ids", "bias", "mask_bits", "row_mask"))
    for b in range(c["B"]):
        base = np.bincount(hist[b, npm[b]:hl[b]], minlength=c["V"]).astype(np.float64)
        prompt = np.zeros(c["V"], bool)
        prompt[hist[b, :min(npm[b], hl[b])]] = True
        add = np.zeros(c["V"])
        if ids is not None:
            np.add.at(add, ids[b][ids[b] >= 0], bias[b][ids[b] >= 0].astype(np.float64))
        for j in range(c["Rj"]):
            n, x = base.copy(), node[b, j]
            while x >= 0:
                n[tok[b, x]] += 1
                x = par[b, x]
            r, y = float(rep[b]), z[b, j]
            hit = prompt | (n > 0)
            y[hit] = np.where(y[hit] > 0, y[hit] / r, y[hit] * r)
            y -= float(freq[b]) * n + float(pres[b]) * (n > 0)
            y += add
            if bits is not None and row_mask[b, j] >= 0:
                w = bits[row_mask[b, j]].view(np.uint8)
                y[np.unpackbits(w, bitorder="little")[:c["V"]] == 0] = -np.inf
    return {"out": torch.from_numpy(z)}
