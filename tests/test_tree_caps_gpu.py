"""Attention of drafted tokens with caps of every size on the GPU, against its float64
definition within the decode tolerance (tests/parity.py)."""
import numpy as np
import pytest

from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.test_tree_gpu import check, env, make, run  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [1.2e-38, 1e-30, 1e-3, 0.7, 300.0, 1e4, 1e5, 1e6, 1e9, 1e20, 2e38, 3e38])
@pytest.mark.parametrize("q_scale", [1.0, 30.0])
def test_caps_of_any_size(env, softcap, q_scale):
    """Caps far above the scores change nothing that can be seen, caps far below them leave their signs."""
    p = make([300, 140], [6, 2], 8, 2, seed=143, q_scale=q_scale)
    p["q"][1, 3] = 0                                          # scores of exactly 0
    check(env, p, softcap=softcap)


def test_capped_scores_that_are_not_finite(env):
    """tanh takes an infinite score to the cap; NaN stays NaN, with the rows that attend it."""
    p = make([140], [6], 8, 2, seed=144)
    p["k"][2, 0, 17] = np.nan
    p["k"][3, 1, 5] = np.inf
    for softcap in (5.0, 1e5):
        got = run(env, p, softcap=softcap)
        with np.errstate(all="ignore"):
            want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"], p["cu"], p["lens"], p["bt"], p["ws"], p["cache"],
                                     softcap=softcap)
        assert np.isnan(want).any() and not np.isnan(want).all()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert_decode_close(got[~np.isnan(want)], want[~np.isnan(want)])
