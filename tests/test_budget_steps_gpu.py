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


@pytest.mark.parametrize("width,n", FORMS)
@pytest.mark.parametrize("group", [4, 8])
def test_scores_of_minus_infinity(env, width, n, group):
    """A key of minus infinity in the workspace (a channel beyond fp16's end) has no weight with the heads
    whose query is positive there. Its warp's other rows are masked, or all the same, or not."""
    for tail, hit in ((1, [0]), (17, [16]), (20, [16, 17, 18, 19]), (33, [3]), (60, list(range(16, 32)))):
        p = _make([256 + tail, tail, 128 + tail][:n], group, 1, seed=103 + tail, width=width)
        p["q"][..., 5] = np.abs(p["q"][..., 5]) + np.float16(0.5)
        p["ws"][:, :, 0, hit, 5] = -np.inf
        _weigh_check(env, _without(p, hit, 0.5), 0.5, got=_weigh(env, p, 0.5))


def _without(p, hit, decay):
    """The inputs without the workspace tokens at `hit`; where none is left, the partial tile's faded weight."""
    stay = [t for t in range(128) if t not in hit]
    ws = np.zeros_like(p["ws"])
    ws[:, :, :, :len(stay)] = p["ws"][:, :, :, stay]
    left = dict(p, lens=p["lens"] - len(hit), ws=ws, w=p["w"].copy())
    for s, length in enumerate(left["lens"]):
        if length % 128 == 0:
            left["w"][s, :, length // 128] *= np.float32(decay)
    return left
