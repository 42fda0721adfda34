"""Decode attention that weighs its tiles for groups of one to eight q-heads (up to four take
another form of the products), at the ends of its operands' ranges."""
import numpy as np
import pytest

from tests.test_budget_gpu import _make, _quantized, _weigh, _weigh_check, env  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
def test_groups(env, preset, group):
    _weigh_check(env, _make([700, 128, 1000, 60], 2 * group, 2, preset, seed=30 + group), decay=0.5)


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("k_mean,k_std,v_mean,v_std", [(0, 1, 1, 0.3), (3, 0.3, 0, 1), (-30, 0.5, 200, 0.5), (0, 3e-4, 0, 3e-4)])
@pytest.mark.parametrize("group", [1, 4])
def test_small_groups_with_tensors_of_any_scale(env, preset, k_mean, k_std, v_mean, v_std, group):
    rng = np.random.default_rng(31)
    p = _make([3 * 128 + 40], group, 1, preset, seed=31)
    k, v = rng.normal(k_mean, k_std, (3, 128, 128)), rng.normal(v_mean, v_std, (3, 128, 128))
    p["cache"], p["bt"] = _quantized(k, v, preset), np.array([[0, 1, 2, -1]], np.int32)
    p["ws"][0, 0, 0], p["ws"][0, 0, 1] = rng.normal(k_mean, k_std, (128, 128)), rng.normal(v_mean, v_std, (128, 128))
    _weigh_check(env, p)


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2"])
@pytest.mark.parametrize("group", [3, 8])
@pytest.mark.parametrize("gap", [10.0, 16.0, 26.0])
def test_heads_and_channels_far_apart(env, preset, group, gap):
    """q-heads 2^gap times one another in one group, keys whose channels are, and a sink: each head's weights by themselves."""
    rng = np.random.default_rng(32)
    p = _make([4 * 128 + 3], group, 1, preset, seed=32)
    k = rng.standard_normal((4, 128, 128)) * np.exp2(np.linspace(-gap / 2, 6, 128))
    v = rng.standard_normal((4, 128, 128))
    k[0, 0] *= 3
    p["cache"], p["bt"] = _quantized(k, v, preset), np.array([[0, 1, 2, 3, -1]], np.int32)
    q = rng.standard_normal((1, group, 128)) * np.exp2(-np.linspace(0, gap, group))[:, None] * 4
    p["q"] = q.astype(np.float16)
    _weigh_check(env, p)


@pytest.mark.parametrize("group", [2, 8])
def test_sums_over_long_flat_rows(env, group):
    """70000 tokens of nearly the same weight."""
    p = _make([70000, 69999], group, 1, "k2v2", seed=33)
    p["q"] = (p["q"] * np.float16(1e-3)).astype(np.float16)
    _weigh_check(env, p)


@pytest.mark.parametrize("group", [4, 8])
def test_what_is_not_finite_stays_with_its_head(env, group):
    p = _make([300, 900], group, 1, seed=34)
    clean = _weigh(env, p)
    p["q"][1, 1] = np.inf
    out, lse, w = _weigh(env, p)
    others = [h for h in range(group) if h != 1]
    assert np.array_equal(out[0], clean[0][0]) and np.array_equal(w[0], clean[2][0])
    assert np.array_equal(out[1, others], clean[0][1, others]) and np.array_equal(lse[1, others], clean[1][1, others])
    assert not np.isfinite(out[1, 1]).any()
