"""Attention of drafted tokens whose weights or values lie far apart, on the GPU, against its
float64 definition within the decode tolerance (tests/parity.py)."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.test_tree_gpu import check, env, make, run  # noqa: F401 (env: the fixture)
from tests.test_tree_range_gpu import quantized

pytestmark = pytest.mark.gpu


def _sink(preset, t, gap, tiles, n_seqs, hkv, group, seed):
    """Sequences of `tiles` tiles whose first token's score is about `gap` above the others', values of mean 1
    behind a first one of nothing; enough of them that a team of the kernel has whole sequences. Shared blocks."""
    rng = np.random.default_rng(seed)
    u = rng.choice([-1.0, 1.0], 128)
    k = 0.05 * rng.standard_normal((3, 128, 128))
    v = 1 + 0.3 * rng.standard_normal((3, 128, 128))
    k[0, 0] += u * gap / 4 * np.sqrt(128) / 128          # a query of 4 u: 4 u . u gap / 4 / sqrt(128) ..
    v[0, 0] = 0
    rec = quantized(k, v, preset)
    p = make([tiles * 128] * n_seqs, [t] * n_seqs, hkv * group, hkv, preset, seed=seed)
    p["cache"] = np.repeat(rec, hkv, axis=1)
    p["bt"] = np.broadcast_to(np.concatenate([[0], 1 + np.arange(tiles - 1) % 2]), (n_seqs, tiles)).astype(np.int32).copy()
    q = 4 * u * (1 + 0.02 * rng.standard_normal((p["n"], hkv * group, 1))) + 0.1 * rng.standard_normal((p["n"], hkv * group, 128))
    p["q"] = q.astype(np.float16)
    p["k"] = (0.3 * rng.standard_normal(p["k"].shape)).astype(np.float16)
    return p


@pytest.mark.parametrize("t,n_seqs", [(1, 60), (8, 40)])          # units of 32 rows, of 64
@pytest.mark.parametrize("gap", [8.0, 12.5, 13.5, 14.5])
@pytest.mark.parametrize("preset", ["k4v2", "k2v2"])
def test_tail_behind_a_sink(env, preset, t, n_seqs, gap):
    p = _sink(preset, t, gap, 128, n_seqs, 8, 8, 150)
    got = run(env, p)
    only = [(0, 0), (n_seqs // 2, 3), (n_seqs - 1, 7)]
    want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"], p["cu"], p["lens"], p["bt"], p["ws"], p["cache"], only=only)
    rows = ~np.isnan(want)
    assert_decode_close(got[rows], want[rows])


@pytest.mark.parametrize("t", [2, 9])
@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
def test_values_of_far_apart_sizes_in_a_tile(env, preset, t):
    """One token of a tile with values a million times the others', and hardly any weight."""
    rng = np.random.default_rng(151)
    u = rng.choice([-1.0, 1.0], 128)
    k = 0.2 * rng.standard_normal((2, 128, 128))
    v = 0.05 * (1 + 0.3 * rng.standard_normal((2, 128, 128)))
    k[:, 40] -= u * 1.5
    v[:, 40] = 50000 * (1 + 0.1 * rng.standard_normal((2, 128)))
    p = make([256], [t], 8, 1, preset, seed=151)
    p["cache"], p["bt"] = quantized(k, v, preset), np.array([[0, 1, -1]], np.int32)
    p["q"] = (2 * u + 0.1 * rng.standard_normal((t, 8, 128))).astype(np.float16)
    p["k"], p["v"] = (0.1 * p["k"]).astype(np.float16), (0.05 * p["v"]).astype(np.float16)
    check(env, p)


@pytest.mark.parametrize("t", [3, 20])
def test_fresh_value_of_great_size_and_little_weight(env, t):
    rng = np.random.default_rng(152)
    u = rng.choice([-1.0, 1.0], 128)
    p = make([50], [t], 8, 1, seed=152)
    p["q"] = (2 * u + 0.1 * rng.standard_normal((t, 8, 128))).astype(np.float16)
    p["k"], p["ws"] = (0.1 * p["k"]).astype(np.float16), (0.1 * p["ws"]).astype(np.float16)
    for x in (p["ws"][0, 0, 0, 7], p["k"][0, 0]):
        x[:] = -u * 0.55                                  # a score 12.4 below the others': 2^-18
    for x in (p["ws"][0, 0, 1, 7], p["v"][0, 0]):
        x[:] = 60000 * rng.choice([-1.0, 1.0], 128)
    check(env, p)
