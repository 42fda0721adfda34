"""Steps of a cache held to a budget that the other tests of these calls leave out: without a workspace,
with rows of scores that are minus infinity, with what a serving loop returns beside its output."""
import numpy as np
import pytest

from tests.test_budget_gpu import _make, _weigh, _weigh_check, env  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu

# table widths and sequences that take each form of the merge: a block a unit with one and with four
# warps a q-head, and a block a q-head
FORMS = [(7, 3), (40, 1), (200, 1)]


@pytest.mark.parametrize("width,n", FORMS)
@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
def test_partial_tile_fades_without_a_workspace(env, width, n, decay):
    """Tokens that are not attended add 0 to their tile; its old weight fades like the others'."""
    kv, _ = env
    p = dict(_make([300, 100, 640][:n], 8, 1, seed=101, width=width), ws=None)
    out, lse, w = _weigh(env, p, decay, expect=kv.FLAG_BAD_LENGTH)
    whole = dict(p, lens=p["lens"] // 128 * 128)
    for s, length in enumerate(p["lens"]):
        if length % 128:
            t = length // 128
            assert np.array_equal(w[s, :, t], decay * p["w"][s, :, t].astype(np.float64))
            w[s, :, t] = p["w"][s, :, t]           # (the definition below has no partial tile)
    _weigh_check(env, whole, decay, got=(out, lse, w))


@pytest.mark.parametrize("width,n", FORMS)
def test_partial_tile_without_a_workspace_beside_what_is_no_number(env, width, n):
    kv, _ = env
    p = dict(_make([300, 140, 640][:n], 8, 1, seed=102, width=width), ws=None)
    p["q"][0, 2] = np.nan
    w = _weigh(env, p, 0.5, expect=kv.FLAG_BAD_LENGTH)[2]
    assert np.isnan(w[0, 0, :2]).all() and np.array_equal(w[0, 0, 2:3], 0.5 * p["w"][0, 0, 2:3].astype(np.float64))
