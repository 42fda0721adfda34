"""Steps of a cache held to a budget that the other tests of these calls leave out: without a workspace,
with scores of minus infinity, with a block that is not there, and with all that a serving loop returns."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import budget_ops as bo
from tests.test_budget_gpu import _make, _weigh, _weigh_check, env  # noqa: F401 (env: the fixture)
from tests.verify_common import record_pool, to_dev

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


@pytest.mark.parametrize("width,n", FORMS)
@pytest.mark.parametrize("group", [4, 8])
def test_a_block_that_is_not_there(env, width, n, group):
    """The tile is left out: outputs, log-sum-exp and weights are those of the other tokens."""
    kv, _ = env
    p = _make([700, 300, 1000][:n], group, 1, seed=104, width=width)
    gone = [(s, t) for s, t in ((0, 2), (0, 4), (2, 0)) if s < n]
    for s, t in gone:
        p["bt"][s, t] = -1 if t else 6             # (the cache has six blocks)
    out, lse, w = _weigh(env, p, 0.5, expect=kv.FLAG_BAD_BLOCK)
    # the definition over each sequence without those tiles, its table and weights without their entries
    for s in range(n):
        lost = [t for t in range(width) if (s, t) in gone]
        mine = [t for t in range(width) if t not in lost]
        assert np.array_equal(w[s][:, lost], 0.5 * p["w"][s][:, lost].astype(np.float64))
        left = dict(p, q=p["q"][s:s + 1], ws=p["ws"][s:s + 1], lens=p["lens"][s:s + 1] - 128 * len(lost),
                    bt=p["bt"][s:s + 1, mine], w=p["w"][s:s + 1][:, :, mine])
        _weigh_check(env, left, 0.5, got=(out[s:s + 1], lse[s:s + 1], w[s:s + 1][:, :, mine]))


@pytest.mark.parametrize("preset,hq", [("k4v2", 8), ("k2v2", 16), ("k4v2l", 4)])
def test_every_output_of_a_serving_loop(env, preset, hq):
    """Append, attention with weights and log-sum-exp, eviction: all outputs of each step against the definitions."""
    kv, torch = env
    hkv, n, width = 2, 3, 7
    rng = np.random.default_rng(62)
    lens = np.array([5 * 128 + 126, 4 * 128 + 127, 125], np.int32)
    pool = record_pool(preset, 6, hkv, 1)
    cache = np.concatenate([pool] * 4)[:n * width]                       # a sequence's own 7 blocks
    bt = np.arange(n * width, dtype=np.int32).reshape(n, width)
    meta = kv.make_meta(hkv, hq, len(cache), width, preset=preset)
    d_cache, d_bt = to_dev(torch, cache), to_dev(torch, bt)
    d_ws = to_dev(torch, synth.workspace_tokens(n, hkv, seed=63))
    d_lens = [to_dev(torch, lens), torch.empty(n, dtype=torch.int32, device="cuda")]
    weights, lse = torch.zeros(n, hkv, width, device="cuda"), torch.empty(n, hq, device="cuda")
    kept = torch.empty(n, hkv, width, dtype=torch.int32, device="cuda")
    budgets = torch.tensor([4, 4, 1], dtype=torch.int32, device="cuda")
    scratch = torch.empty(kv.decode_weights_scratch_bytes(meta, n), dtype=torch.uint8, device="cuda")
    out = torch.empty(n, hq, 128, dtype=torch.float16, device="cuda")
    for step in range(4):
        q, k, v = (torch.tensor(rng.standard_normal((n, h, 128)), dtype=torch.float16).cuda() for h in (hq, hkv, hkv))
        kv.kvarn_append_decode(k, v, d_lens[0], d_lens[1], d_bt, d_ws, d_cache, meta)
        before = weights.cpu().numpy()
        kv.kvarn_decode_attention_weights(q, d_cache, d_ws, d_bt, d_lens[1], weights, out, scratch, meta, decay=0.75, lse=lse)
        torch.cuda.synchronize()
        held, ln, c = weights.cpu().numpy(), d_lens[1].cpu().numpy(), d_cache.cpu().numpy()
        p = dict(q=q.cpu().numpy(), cache=c, ws=d_ws.cpu().numpy(), bt=bt, lens=ln, w=before, preset=preset)
        _weigh_check(env, p, 0.75, got=(out.double().cpu().numpy(), lse.double().cpu().numpy(), held.astype(np.float64)))
        kv.kvarn_evict_tiles(weights, weights, d_lens[1], d_lens[0], d_bt, budgets, kept, d_cache, meta)
        torch.cuda.synchronize()
        want = bo.evict_tiles(held, ln, bt, budgets.cpu().numpy(), c, 1, 1)
        for a, b in zip((kept, d_lens[0], weights, d_cache), want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert kv.kvarn_device_flags() == 0
