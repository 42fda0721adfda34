"""Shared by the tests of the calls around a verify step: oracle-quantized tiles in a
paged layout, random trees, and the roundings that tolerances count."""
from __future__ import annotations

import functools

import numpy as np

import kvarn_synth as synth
from oracle import kvarn_oracle as o

HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
TINY = {"float16": 2.0 ** -25, "bfloat16": 2.0 ** -134, "float32": 2.0 ** -150}   # half a subnormal step


@functools.lru_cache(maxsize=None)
def record_pool(preset: str, n: int, hkv: int, seed: int) -> np.ndarray:
    """n blocks of oracle-quantized tiles, uint8 [n, hkv, record bytes]."""
    k, v = synth.prefill_kv(n * 128, hkv, seed=seed)
    k = k.reshape(n, 128, hkv, 128).swapaxes(1, 2)
    v = v.reshape(n, 128, hkv, 128).swapaxes(1, 2)
    rec, _, _ = o.quantize_tiles(k, v, preset=preset)
    return rec


def paged(preset, lens, hkv, seed, pool=6, width=None):
    """cache, block tables (the pool's blocks over and over, in a random order: blocks may
    be shared) and workspace for the given lengths. Unused table entries are -1."""
    g = np.random.default_rng(seed)
    cache = record_pool(preset, pool, hkv, seed % 3)
    width = width or max(1, max(int(n) // 128 for n in lens) + 1)
    bt = np.full((len(lens), width), -1, np.int32)
    for s, n in enumerate(lens):
        full = min(int(n) // 128, width)
        bt[s, :full] = g.integers(0, pool, full)
    ws = synth.workspace_tokens(len(lens), hkv, seed=seed)
    return cache, bt, ws


def random_tree(n, rng, chain=False):
    """Ancestor words (Python ints, own bit set) and depths of a random tree of n tokens."""
    words, depths = [], []
    for p in range(n):
        up = p - 1 if chain else int(rng.integers(max(-1, p // 2 - 2), p)) if p else -1
        words.append((words[up] if up >= 0 else 0) | 1 << p)
        depths.append(depths[up] + 1 if up >= 0 else 0)
    return words, depths


def to_dev(torch, a, device="cuda"):
    a = np.ascontiguousarray(a)
    if a.dtype == np.float16:
        return torch.from_numpy(a.view(np.int16)).view(torch.float16).to(device)
    return torch.from_numpy(a).to(device)


def words_to_dev(torch, words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")
