"""Float64 CPU definitions of the calls around a cache held to a budget: rotation along
several axes, decode attention with its log-sum-exp and each tile's weight, and the
eviction of tiles. Plain loops over the cache's own oracle; shares no code with the CUDA
library.
"""
from __future__ import annotations

import numpy as np

from . import kvarn_oracle as o
from .verify_ops import cached_tokens, qk_norm_rope

B, D = o.B, o.D


def qk_norm_rope_axes(x, weight, eps, inv_freq, positions, axes, interleaved):
    """x [n, heads, 128], positions [n_axes, n], axes: each pair's; float64 [n, heads, 128]."""
    out = qk_norm_rope(x, weight, eps, None, None, interleaved)
    half = len(inv_freq)
    normed = out.copy()
    for a in sorted(set(axes)):
        turned = qk_norm_rope(normed, None, eps, inv_freq, positions[a], interleaved)
        for i in (i for i in range(half) if axes[i] == a):
            for ch in ((2 * i, 2 * i + 1) if interleaved else (i, i + half)):
                out[..., ch] = turned[..., ch]
    return out


def decode_weights(q, cache, workspace, block_tables, seq_lens, weights, decay=1.0, pairs=None):
    """Returns (out [n, Hq, 128], lse [n, Hq], weights [n, Hkv, max_blocks]), float64."""
    n, hq, _ = q.shape
    hkv = cache.shape[1]
    g = hq // hkv
    out, lse = np.zeros(q.shape), np.full((n, hq), -np.inf)
    weights = np.array(weights, np.float64)
    for s, h in pairs if pairs is not None else [(s, h) for s in range(n) for h in range(hkv)]:
        length = int(seq_lens[s])
        if length <= 0:
            continue
        k, v = cached_tokens(cache, workspace, block_tables[s], s, length, h)
        x = np.asarray(q[s, h * g:(h + 1) * g], np.float64) @ k.T / np.sqrt(D)
        top = x.max(1, keepdims=True)
        e = np.exp(x - top)
        total = e.sum(1, keepdims=True)
        out[s, h * g:(h + 1) * g] = e @ v / total
        lse[s, h * g:(h + 1) * g] = (top + np.log(total))[:, 0]
        p = (e / total).sum(0)
        for t in range(-(-length // B)):
            if t < weights.shape[2]:
                old = decay * weights[s, h, t] if decay else 0.0
                weights[s, h, t] = old + p[t * B:(t + 1) * B].sum()
    return out, lse, weights


def score_error(q, cache, workspace, block_tables, seq_lens, s, h, preset):
    """A bound on the error of an fp32 evaluation of the natural-log scores of unit (s, h), whose
    products take 22 bits of each factor: the sums run over 128 channels in steps of
    16 (8 roundings, hi and lo parts, of at most 2^-23), the zero points' sum has
    below 24 roundings, and the rotated query is a sum of 7 levels."""
    g = q.shape[1] // cache.shape[1]
    qh = np.asarray(q[s, h * g:(h + 1) * g], np.float64)
    qr = np.abs(o.rotate(qh.T).T)
    kb, _ = o.PRESETS[preset]
    length, worst = int(seq_lens[s]), 0.0
    flat = np.abs(qh).sum(1) / np.sqrt(D)               # no channel of the rotated query is above it
    for t in range(length // B):
        gk, _ = o.unpack_record(cache[int(block_tables[s][t]), h])
        size = gk["r"] * ((2 ** kb - 1) * np.abs(gk["s"]) + np.abs(gk["z"]))
        m = (qr @ size).max() * gk["c"].max() / np.sqrt(D)
        m7 = flat.max() * size.sum() * gk["c"].max() / np.sqrt(D)
        worst = max(worst, 2.0 ** -24 * (64 * m + 8 * m7))
    if length % B:
        k = np.abs(np.asarray(workspace[s, h, 0, :length % B], np.float64))
        worst = max(worst, 2.0 ** -24 * 32 * (np.abs(qh) @ k.T).max() / np.sqrt(D))
    return worst


def evict_tiles(weights, seq_lens, block_tables, budgets, cache, keep_first, keep_last):
    """Returns (kept int32, lengths int32, weights float32, cache). Sequences that are longer than
    their table, or whose blocks are not all there, stay as they are."""
    weights, cache = np.array(weights, np.float32), np.array(cache, copy=True)
    n_seqs, hkv, width = weights.shape
    kept = np.full(weights.shape, -1, np.int32)
    lens = np.array(seq_lens, np.int32)
    out = weights.copy()
    for s in range(n_seqs):
        tiles = max(int(seq_lens[s]), 0) // B
        n = min(tiles, width)
        b = n if budgets[s] < 0 else min(n, int(budgets[s]))
        blocks = [int(x) for x in block_tables[s][:n]]
        if tiles > width or (b < n and any(not 0 <= x < cache.shape[0] for x in blocks)):
            kept[s, :, :n] = np.arange(n)
            continue
        first = min(keep_first, b)
        last = min(keep_last, b - first)
        for h in range(hkv):
            w = weights[s, h]
            rank = sorted(range(first, n - last), key=lambda t: (np.isnan(w[t]), 0.0 if np.isnan(w[t]) else -w[t], t))
            chosen = set(rank[:b - first - last])
            gone = [t for t in range(first, n - last) if t not in chosen]
            late = [t for t in sorted(chosen) if t >= b - last]
            slots = []
            for t in range(b - last):
                slots.append(t if t < first or t in chosen else late.pop(0))
            slots += range(n - last, n)
            kept[s, h, :n] = slots + gone
            old = cache[:, h].copy()
            for t, src in enumerate(slots):
                if src != t:
                    cache[blocks[t], h] = old[blocks[src]]
            row = [w[t] for t in slots] + ([w[n]] if n < width else [])
            out[s, h] = 0
            out[s, h, :len(row)] = row
        lens[s] -= 128 * (n - b)
    return kept, lens, out, cache
