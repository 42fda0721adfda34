"""Float64 CPU definitions of the calls around a verify step: norm and rotation of
projected rows, attention of drafted tokens over the quantized cache, the append of
several tokens, and the reading back of cached tokens. Plain loops over the cache's
own oracle; shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np

from . import kvarn_oracle as o

B, D = o.B, o.D


def qk_norm_rope(x, weight, eps, inv_freq, positions, interleaved):
    """x [n, heads, 128] (any float type), weight [128] or None, inv_freq float32
    [rotary / 2] or None; returns float64 [n, heads, 128]."""
    x = np.asarray(x, np.float64).copy()
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if inv_freq is None:
        return x
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        # whole turns taken out in integers: freq / 2 pi as a fraction of 2^80
        f = int(np.float64(inv_freq[i]) / (2 * np.pi) * 2.0 ** 80)
        t = np.array([((int(p) * f) % (1 << 80)) / 2.0 ** 80 for p in positions])[:, None] * 2 * np.pi
        xa, xb = x[..., a].copy(), x[..., b].copy()
        x[..., a] = xa * np.cos(t) - xb * np.sin(t)
        x[..., b] = xb * np.cos(t) + xa * np.sin(t)
    return x


def cached_tokens(cache, workspace, block_table, seq, seq_len, head):
    """K and V [seq_len, 128] of one sequence and kv-head, float64."""
    n_full, n_ws = int(seq_len) // B, int(seq_len) % B
    ks, vs = [np.zeros((0, D))], [np.zeros((0, D))]
    if n_full:
        kh, vh = o.dequant_record(cache[np.asarray(block_table[:n_full], np.int64), head])
        ks.append(np.swapaxes(kh, -1, -2).reshape(-1, D))
        vs.append(np.swapaxes(vh, -1, -2).reshape(-1, D))
    if n_ws:
        ks.append(np.asarray(workspace[seq, head, 0, :n_ws], np.float64))
        vs.append(np.asarray(workspace[seq, head, 1, :n_ws], np.float64))
    return np.concatenate(ks), np.concatenate(vs)


def tree_attention(q, k_new, v_new, masks, cu, seq_lens, block_tables, workspace, cache, positions=None, scale=0.0,
                   softcap=0.0, window=0, slopes=None, only=None):
    """masks: Python ints, one a new token (bit j: the sequence's j-th new token), or None
    (a chain). Returns float64 [n_tokens, Hq, 128]; rows outside `only` (a list of
    (sequence, kv-head) pairs) and outside every sequence are NaN."""
    n, hq, _ = q.shape
    hkv = k_new.shape[1]
    g = hq // hkv
    out = np.full(q.shape, np.nan)
    for s in range(len(seq_lens)):
        a, b = int(cu[s]), int(cu[s + 1])
        length = int(seq_lens[s])
        for h in range(hkv):
            if a == b or (only is not None and (s, h) not in only):
                continue
            k, v = cached_tokens(cache, workspace, block_tables[s], s, length, h)
            k = np.concatenate([k, np.asarray(k_new[a:b, h], np.float64)])
            v = np.concatenate([v, np.asarray(v_new[a:b, h], np.float64)])
            for t in range(a, b):
                word = (1 << (t - a + 1)) - 1 if masks is None else int(masks[t])
                seen = np.array([True] * length + [bool(word >> j & 1) for j in range(b - a)])
                x = np.asarray(q[t, h * g:(h + 1) * g], np.float64) @ k.T * (scale or 1 / np.sqrt(D))
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if window or slopes is not None:
                    pk = np.concatenate([np.arange(length), np.asarray(positions[a:b], np.int64)])
                    gap = int(positions[t]) - pk
                    if slopes is not None:
                        x = x - np.asarray(slopes, np.float64)[h * g:(h + 1) * g, None] * gap
                    if window:
                        seen = seen & (gap < window)
                if not seen.any():
                    out[t, h * g:(h + 1) * g] = 0
                    continue
                x = x[:, seen]
                p = np.exp(x - x.max(-1, keepdims=True))
                out[t, h * g:(h + 1) * g] = p / p.sum(-1, keepdims=True) @ v[seen]
    return out


def append_tokens(k_new, v_new, cu, seq_lens, block_tables, workspace, cache, accepted=None, n_accepted=None):
    """Returns (workspace, cache, lengths, completed), completed = [(sequence, block, tile
    of fp16 rows [Hkv, 2, 128, 128])]."""
    ws, cache = np.array(workspace, copy=True), np.array(cache, copy=True)
    preset = o.layout_of(cache.shape[-1]).name
    lens, done = np.array(seq_lens, copy=True), []
    for s in range(len(lens)):
        n = int(cu[s + 1]) - int(cu[s]) if accepted is None else int(n_accepted[s])
        for i in range(n):
            r = int(cu[s]) + (i if accepted is None else int(accepted[s, i]))
            pos = int(lens[s]) % B
            ws[s, :, 0, pos], ws[s, :, 1, pos] = k_new[r], v_new[r]
            if pos == B - 1:
                blk = int(block_tables[s, int(lens[s]) // B])
                done.append((s, blk, ws[s].copy()))
                cache[blk] = o.quantize_tiles(ws[s, :, 0], ws[s, :, 1], preset=preset)[0]
            lens[s] += 1
    return ws, cache, lens, done


def read_tokens(cache, workspace, block_tables, seq_lens, first, cu):
    """K and V float64 [n_tokens, Hkv, 128]."""
    hkv = cache.shape[1]
    k = np.full((int(cu[-1]), hkv, D), np.nan)
    v = k.copy()
    for s in range(len(seq_lens)):
        f, n = int(first[s]), int(cu[s + 1]) - int(cu[s])
        for h in range(hkv):
            ks, vs = cached_tokens(cache, workspace, block_tables[s], s, seq_lens[s], h)
            k[cu[s]:cu[s + 1], h], v[cu[s]:cu[s + 1], h] = ks[f:f + n], vs[f:f + n]
    return k, v


def read_magnitude(cache, workspace, block_tables, seq_lens, first, cu, preset):
    """Per output row and kv-head: sum over channels of the largest magnitude that the
    dequantized row's terms can have, over sqrt(128) (0 for workspace rows): the scale of
    an fp32 evaluation's error. Array [2 (K, V), n_tokens, Hkv]."""
    hkv = cache.shape[1]
    kb, vb = o.PRESETS[preset]
    out = np.zeros((2, int(cu[-1]), hkv))
    for s in range(len(seq_lens)):
        for j in range(int(cu[s + 1]) - int(cu[s])):
            t = int(first[s]) + j
            if t // B >= int(seq_lens[s]) // B:
                continue
            for h in range(hkv):
                gk, gv = o.unpack_record(cache[int(block_tables[s][t // B]), h])
                at = t % B
                m = (gk["r"] * (2 ** kb * gk["s"] + np.abs(gk["z"]))).sum() * gk["c"][at]
                out[0, int(cu[s]) + j, h] = m / np.sqrt(D)
                m = gv["r"].sum() * gv["c"][at] * (2 ** vb * gv["s"][at] + abs(gv["z"][at]))
                out[1, int(cu[s]) + j, h] = m / np.sqrt(D)
    return out
