"""Attention of drafted tokens at the ends of its operands' ranges on the GPU, against its
float64 definition within the decode tolerance (tests/parity.py)."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.test_tree_gpu import check, env, make, run  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


def quantized(k, v, preset):
    """Tiles [n, tokens, 128] of one kv-head as a cache of n blocks."""
    return o.quantize_tiles(np.asarray(k, np.float16)[:, None], np.asarray(v, np.float16)[:, None], preset=preset)[0]


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size,noise,q_size,q_noise", [
    (5.0, 0.0, 12.0, 0.1), (1.9, 0.0, 1.9, 0.0), (24.0, 0.01, 30.0, 0.0), (250.0, 0.1, 12.0, 0.1), (6000.0, 1.0, 1.5, 0.0),
    (15.9, 0.0, 15.9, 0.0),
])
def test_keys_constant_in_one_channel(env, preset, sign, size, noise, q_size, q_noise):
    """Keys that are (nearly) the same number in one channel and nothing elsewhere, under queries
    along that channel: flat after the rotation, so that the zero points of all 128 channels add up with one
    sign, and far above the tile's steps."""
    rng = np.random.default_rng(140)
    p = make([300], [9], 8, 1, preset, seed=140)
    _, v = synth.prefill_kv(2 * 128, 1, seed=141)
    k = noise * rng.standard_normal((2, 128, 128))
    k[..., 5] += sign * size
    p["cache"], p["bt"] = quantized(k, v.reshape(2, 128, 128), preset), np.array([[0, 1, -1]], np.int32)
    q = q_noise * rng.standard_normal((9, 8, 128))
    q[..., 5] += q_size
    p["q"] = q.astype(np.float16)
    check(env, p)


def _kept(p, keep, scores):
    """The definition over one sequence and kv-head of which only the cached tokens `keep` are there, at their own
    positions: scores(query row, head, keys, gaps) -> scores, -inf where masked."""
    n, hq, _ = p["q"].shape
    k, v = vo.cached_tokens(p["cache"], p["ws"], p["full_bt"][0], 0, p["lens"][0], 0)
    out = np.zeros(p["q"].shape)
    for t in range(n):
        mine = [j for j in range(n) if p["words"][t] >> j & 1]
        kk = np.concatenate([k[keep], p["k"][mine, 0].astype(np.float64)])
        vv = np.concatenate([v[keep], p["v"][mine, 0].astype(np.float64)])
        gap = int(p["pos"][t]) - np.concatenate([keep, p["pos"][mine].astype(np.int64)])
        for m in range(hq):
            x = scores(p["q"][t, m].astype(np.float64), m, kk, gap)
            if np.isfinite(x).any():
                w = np.exp(x - x.max())
                out[t, m] = w / w.sum() @ vv
    return out


@pytest.mark.parametrize("score", [dict(window=200), dict(window=45), dict(slopes=[0.5, 0.02, 0.0, 0.11]),
                                   dict(window=150, slopes=[0.01, 0.3, 0.0, 0.05])])
@pytest.mark.parametrize("t", [3, 17])
def test_positions_behind_a_short_table(env, t, score):
    """Of a sequence longer than its block table the tiles behind the table are left out; its workspace tokens keep
    their positions."""
    kv, _ = env
    p = make([5 * 128 + 60], [t], 4, 1, seed=142)
    p["full_bt"], p["bt"] = p["bt"], p["bt"][:, :2].copy()
    got = run(env, p, expect=kv.FLAG_BAD_LENGTH, **score)
    slopes, window = np.array(score.get("slopes", [0.0] * 4)), score.get("window", 1 << 40)
    keep = np.concatenate([np.arange(256), np.arange(640, 700)])
    want = _kept(p, keep, lambda q, m, k, gap: np.where(gap < window, k @ q / np.sqrt(128) - slopes[m] * gap, -np.inf))
    assert_decode_close(got, want)


def _extreme(preset, t, size, seed):
    """Keys of `size` in the cache, the workspace and the drafted tokens, values of about 1."""
    rng = np.random.default_rng(seed)
    p = make([256 + 40], [t], 8, 1, preset, seed=seed)

    def keys(*shape):
        return (size * rng.standard_normal(shape + (128,))).clip(-6e4, 6e4).astype(np.float16)

    p["cache"] = quantized(keys(2, 128), rng.standard_normal((2, 128, 128)), preset)
    p["bt"] = np.array([[0, 1, -1]], np.int32)
    p["ws"][0, 0, 0, :40], p["ws"][0, 0, 1, :40] = keys(40), rng.standard_normal((40, 128))
    p["k"], p["v"] = keys(t, 1), rng.standard_normal((t, 1, 128)).astype(np.float16)
    return p, rng


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("t", [2, 4, 9])
@pytest.mark.parametrize("big,small,size", [(3e3, 3e-2, 1e2), (3e4, 3e-2, 1e2), (3e4, 3e-3, 1e3)])
def test_query_rows_far_apart(env, preset, t, big, small, size):
    """One row of q up to ten million times the others of its sequence and kv-head, and keys that give the others
    scores of about 3."""
    p, rng = _extreme(preset, t, size, 145)
    q = small * rng.standard_normal((t, 8, 128))
    q[t // 2, 3] = big / 3 * np.clip(rng.standard_normal(128), -3, 3)
    p["q"] = q.astype(np.float16)
    check(env, p)
    check(env, p, window=250)


@pytest.mark.parametrize("preset", ["k4v2", "k2v2"])
@pytest.mark.parametrize("t", [2, 4, 9, 40])
@pytest.mark.parametrize("lens", [296, 256, 40, 0])
def test_scores_beyond_what_is_added_exactly(env, preset, t, lens):
    """Scores of 10^8 to 10^9, whose neighbours in fp32 are 64 apart: the largest key of a row takes all its weight."""
    p, rng = _extreme(preset, t, 2e4, 146)
    p["lens"] = np.array([lens], np.int32)
    p["q"] = (5e4 / 3 * np.clip(rng.standard_normal((t, 8, 128)), -3, 3)).astype(np.float16)
    if lens % 128 == 0:
        p["ws"][:] = 0
    elif lens < 128:
        p["bt"][:] = -1
    p["pos"] = (lens + np.arange(t)).astype(np.int32)
    check(env, p)
    check(env, p, window=250)
