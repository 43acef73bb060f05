"""CPU oracle of the 8-bit KV cache, the page planner and the logits
adjustment (test infrastructure; float64 numpy, no code shared with the CUDA
path).

A cache here is a pair ``codes`` float64 [n_pages][Hkv][2][page_size][d] (the
values of the e4m3 codes) and ``scales`` float64 [n_pages][Hkv][2]; the
element is code * scale.  The steps follow the definitions in the header of
the C boundary: one scale per (page, head) for keys and one for values, the
smallest power of two within 2^-60 .. 2^60 that holds the block's values in
448 steps, growing only while a page fills.
"""

from __future__ import annotations

import math

import numpy as np

E_MIN, E_MAX = -60, 60


def e4m3_table():
    """Value of each of the 256 e4m3 codes (4 exponent bits, bias 7, 3
    mantissa bits; 0x7f and 0xff are NaN, no infinities)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-v if s else v)
    return out


def round_e4m3(x):
    """Nearest e4m3 value, ties to the even code, saturating at 448; a
    non-finite input is NaN."""
    x = np.asarray(x, dtype=np.float64)
    pos = e4m3_table()[:127]                     # increasing, code = index
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.searchsorted(pos, a)                 # pos[hi - 1] < a <= pos[hi]
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isfinite(x), np.copysign(pos[pick], x), np.nan)


def block_exponent(amax):
    """Smallest e in [-60, 60] with amax <= 448 * 2^e (60 where none is)."""
    for e in range(E_MIN, E_MAX):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def write_rows(codes, scales, page, first, rows_k, rows_v):
    """New rows [n][Hkv][d] into one page at offsets first .. (in place); a
    row given as None leaves its slot alone."""
    for x, rows in ((0, rows_k), (1, rows_v)):
        for h in range(codes.shape[1]):
            new = [(first + i, np.asarray(r[h], dtype=np.float64)) for i, r in enumerate(rows)
                   if r is not None]
            if not new:
                continue
            vals = np.concatenate([r for _, r in new])
            fin = np.abs(vals[np.isfinite(vals)])
            s = 2.0 ** block_exponent(fin.max() if fin.size else 0.0)
            bad = not np.isfinite(vals).all()
            if first > 0:
                was = scales[page, h, x]
                if np.isnan(was):
                    bad = True
                else:
                    if s > was:
                        old = codes[page, h, x, :first]
                        codes[page, h, x, :first] = round_e4m3(old * (was / s))
                    s = max(s, was)
            for t, r in new:
                codes[page, h, x, t] = round_e4m3(r / s)
            scales[page, h, x] = math.nan if bad else s


def commit(codes, scales, page_table, seq_len, free_pages, free_head, k_block, v_block, paths,
           page_size):
    """kv_commit into the 8-bit cache; returns copies (codes, scales,
    page_table, seq_len, free_head).  Blocks [B][Hkv][R][d]."""
    codes, scales = codes.copy(), scales.copy()
    table, seq = page_table.copy(), seq_len.copy()
    for b, path in enumerate(paths):
        i = 0
        while i < len(path):
            pos = int(seq[b]) + i
            if pos % page_size == 0:
                table[b, pos // page_size] = free_pages[free_head]
                free_head += 1
            n = min(page_size - pos % page_size, len(path) - i)
            rk = [k_block[b][:, r] for r in path[i:i + n]]
            rv = [v_block[b][:, r] for r in path[i:i + n]]
            write_rows(codes, scales, table[b, pos // page_size], pos % page_size, rk, rv)
            i += n
        seq[b] += len(path)
    return codes, scales, table, seq, free_head


def append(codes, scales, k, v, slot_map, page_size):
    """Packed rows [n][Hkv][d] into their slots; returns copies."""
    codes, scales = codes.copy(), scales.copy()
    i, n = 0, len(slot_map)
    while i < n:
        if slot_map[i] < 0:
            i += 1
            continue
        page, off = divmod(int(slot_map[i]), page_size)
        m = 1
        while i + m < n and off + m < page_size and slot_map[i + m] in (-1, slot_map[i] + m):
            m += 1
        keep = [slot_map[i + t] >= 0 for t in range(m)]
        write_rows(codes, scales, page, off, [r if w else None for r, w in zip(k[i:i + m], keep)],
                   [r if w else None for r, w in zip(v[i:i + m], keep)])
        i += m
    return codes, scales


def gather(codes, scales, page_table, seq_len):
    """Per-request prefix K and V [Hkv][S][d] as values."""
    ps = codes.shape[3]
    val = codes * scales[:, :, :, None, None]
    out = []
    for b, S in enumerate(seq_len):
        pages = page_table[b, :-(-int(S) // ps)]
        x = val[pages].transpose(2, 1, 0, 3, 4).reshape(2, codes.shape[1], -1, codes.shape[4])
        out.append(x[:, :, :int(S)])
    return [x[0] for x in out], [x[1] for x in out]


def page_plan(seq_len, n_new, page_table, free_pages, free_head, page_size, n_slots):
    """(page_table, free_head, cu_new, slot_map, new_len): pages in list
    order, requests in ascending order; requests over their table's capacity
    get no slots; none do when the list is too short."""
    table = page_table.copy()
    B, cap = len(seq_len), page_table.shape[1] * page_size
    cu = np.zeros(B + 1, dtype=np.int32)
    slots = np.full(n_slots, -1, dtype=np.int64)
    new_len = np.array(seq_len, dtype=np.int32).copy()
    ok = [0 <= s and 0 <= n and s + n <= cap for s, n in zip(seq_len, n_new)]
    need = sum(-(-(int(s) + int(n)) // page_size) - -(-int(s) // page_size)
               for s, n, k in zip(seq_len, n_new, ok) if k)
    serve = free_head >= 0 and free_head + need <= len(free_pages)
    for b in range(B):
        n = max(0, int(n_new[b]))
        cu[b + 1] = cu[b] + n
        if not (ok[b] and serve):
            continue
        for i in range(n):
            pos = int(seq_len[b]) + i
            if pos % page_size == 0:
                table[b, pos // page_size] = free_pages[free_head]
                free_head += 1
            if cu[b] + i < n_slots:
                slots[cu[b] + i] = int(table[b, pos // page_size]) * page_size + pos % page_size
        new_len[b] += n
    return table, free_head, cu, slots, new_len


def logits_adjust(logits, history, n_prompt, tokens, tree_parent, row_node, repetition, presence,
                  frequency, biases, masks, row_mask):
    """Adjusted logits [B][Rj][V] (float64).  history: list of token lists;
    biases: list of (id, value) lists; masks: bool [n][V]; row_node -1 and
    row_mask < 0: none."""
    out = np.array(logits, dtype=np.float64)
    B, Rj, V = out.shape
    for b in range(B):
        for j in range(Rj):
            n = {}
            for i, t in enumerate(history[b]):
                if 0 <= t < V:
                    n[t] = n.get(t, 0) + int(i >= n_prompt[b])
            x = int(row_node[b][j])
            while x >= 0:
                t = int(tokens[b][x])
                if 0 <= t < V:
                    n[t] = n.get(t, 0) + 1
                x = int(tree_parent[b][x])
            z = out[b, j]
            for v, k in n.items():
                z[v] = z[v] / repetition[b] if z[v] > 0 else z[v] * repetition[b]
                z[v] -= frequency[b] * k + (presence[b] if k else 0.0)
            for t, x in biases[b]:
                if 0 <= t < V:
                    z[t] += x
            if masks is not None and row_mask[b][j] >= 0:
                z[~masks[row_mask[b][j]]] = -math.inf
    return out
