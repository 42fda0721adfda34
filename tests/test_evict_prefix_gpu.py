"""Eviction behind a long prefix that stays (keep_first), on tables of more tiles than keys are held
in shared memory (10240): the tiles to choose from lie before, across and behind that slot."""
import numpy as np
import pytest

from tests.test_budget_gpu import _evict, _tiles, env  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tiles,first,last,budget", [
    (11000, 10700, 0, 10900),       # all to choose from behind slot 10240: one warp's search
    (11000, 10700, 3, 10999),       # the smallest ones first
    (12000, 11000, 500, 11800),
    (10400, 10000, 2, 10200),       # across it, one warp
    (10400, 10000, 2, 10398),
    (10500, 9900, 260, 10300),      # the last of them at slot 10239
    (10500, 9729, 259, 10300),      # 512 of them, the last at slot 10240
    (10500, 9729, 258, 10300),      # 513
    (12000, 10500, 2, 11000),       # behind it, the whole block's search
    (12000, 9000, 2, 11990),        # across it
    (22000, 500, 0, 700),           # more to choose from than are held
    (22000, 11000, 5, 21990),
])
def test_evict_behind_a_long_prefix(env, tiles, first, last, budget, in_place):
    w, lens, bt, cache = _tiles([tiles], 1, seed=first + last)
    _evict(env, w, lens, bt, [budget], cache, first, last, in_place=in_place)


def test_evict_ties_behind_a_long_prefix(env):
    w, lens, bt, cache = _tiles([10700, 10400], 1, seed=7)
    w[:] = np.random.default_rng(7).integers(0, 3, w.shape)
    w[..., 5::7] = np.nan
    for first, budget in ((10300, 10350), (10000, 10200), (9000, 10300)):
        _evict(env, w, lens, bt, [budget, budget], cache, first, 1)
