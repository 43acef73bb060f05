"""CPU oracle of a prompt chunk's way through the cache: rotary positions, the
writer of the cache of rows, and the chunk's attention (test infrastructure;
float64 numpy, no code shared with the CUDA path)."""

from __future__ import annotations

import math

import numpy as np


def rope_freqs(rot, base, kind="plain", factor=1.0, trained_len=0.0, low=0.0, high=0.0):
    """Radians a position of each pair, one by one."""
    out = []
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        if kind == "linear":
            f = f / factor
        elif kind == "ramp":
            turns = trained_len / (2 * math.pi / f)
            if turns <= low:
                f = f / factor
            elif turns < high:
                w = (turns - low) / (high - low)
                f = w * f + (1 - w) * f / factor
        out.append(f)
    return np.array(out)


def rope(x, positions, freqs, layout, attention=1.0):
    """x [n][H][d]; a negative position leaves its row as it is."""
    out = np.array(x, dtype=np.float64)
    half = len(freqs)
    for t, pos in enumerate(positions):
        if pos < 0:
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + half)
            angle = float(pos) * float(freqs[i])
            c, s = attention * math.cos(angle), attention * math.sin(angle)
            u, w = out[t, :, a].copy(), out[t, :, b].copy()
            out[t, :, a], out[t, :, b] = u * c - w * s, w * c + u * s
    return out


def append_rows(k_cache, v_cache, k, v, slot_map, paged):
    """Packed rows [n][Hkv][d] into copies of a paged cache [P][H][d / 64][ps][64]
    or a contiguous one [B][H][max_seq][d]."""
    kc, vc = k_cache.copy(), v_cache.copy()
    for i, slot in enumerate(slot_map):
        if slot < 0:
            continue
        block, t = divmod(int(slot), kc.shape[3] if paged else kc.shape[2])
        for cache, rows in ((kc, k), (vc, v)):
            for h in range(rows.shape[1]):
                if paged:
                    cache[block, h, :, t] = rows[i, h].reshape(-1, 64)
                else:
                    cache[block, h, t] = rows[i, h]
    return kc, vc


def chunk_attention(q, keys, values, seq_len, cu_new, scale=None):
    """q [n][Hq][d]; keys, values: per request [Hkv][seq_len + new][d].  Returns
    o and lse [n][Hq], NaN in rows that belong to no request, and the sums of
    weight * |value| and the largest |q| . |k| scale of each row (what error
    bounds need).  A row's hidden tokens take no part; a token's weight is 0
    where its score is -inf."""
    n, Hq, d = q.shape
    scale = scale or 1 / math.sqrt(d)
    q = np.asarray(q, dtype=np.float64)
    o = np.full(q.shape, np.nan)
    lse, big = np.full((n, Hq), np.nan), np.zeros((n, Hq))
    mag = np.full(q.shape, np.nan)
    with np.errstate(invalid="ignore", over="ignore"):
        for b in range(len(keys)):
            G = Hq // keys[b].shape[0] if len(keys[b]) else 1
            for i in range(int(cu_new[b + 1]) - int(cu_new[b])):
                row, seen = int(cu_new[b]) + i, int(seq_len[b]) + i + 1
                for h in range(Hq):
                    k = np.asarray(keys[b][h // G][:seen], dtype=np.float64)
                    v = np.asarray(values[b][h // G][:seen], dtype=np.float64)
                    s = k @ q[row, h] * scale
                    if np.isnan(s).any() or np.isposinf(s).any():
                        o[row, h] = mag[row, h] = lse[row, h] = np.nan
                        continue
                    if np.isneginf(s).all():
                        o[row, h] = mag[row, h] = 0.0
                        lse[row, h] = -np.inf
                        continue
                    lse[row, h] = np.logaddexp.reduce(s)
                    p = np.exp(s - lse[row, h])
                    o[row, h], mag[row, h] = p @ v, p @ np.abs(v)
                    big[row, h] = (np.abs(k) @ np.abs(q[row, h])).max() * scale
    return o, lse, mag, big
