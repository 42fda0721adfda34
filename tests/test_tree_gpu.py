"""Attention of drafted tokens over the quantized cache on the GPU, against its float64
definition, within the decode tolerance (tests/parity.py)."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.verify_common import paged, random_tree, to_dev, words_to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import kv_cache_quantization_x128_gb300 as kv
    torch.cuda.set_device(0)
    kv.kvarn_device_flags()
    return kv, torch


def make(lens, counts, hq, hkv, preset="k4v2", seed=70, chain=False, words=None, q_scale=1.0):
    rng = np.random.default_rng(seed)
    cache, bt, ws = paged(preset, lens, hkv, seed)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(cu[-1])
    q = (synth.queries(n, hq, seed) * np.float16(q_scale)).astype(np.float16)
    k, v = synth.prefill_kv(n, hkv, seed=seed + 1)
    trees = [random_tree(c, rng, chain) for c in counts]
    pos = np.array([lens[s] + d for s in range(len(lens)) for d in trees[s][1]], np.int32)
    return dict(lens=np.asarray(lens, np.int32), cu=cu, cache=cache, bt=bt, ws=ws, q=q, k=k, v=v, pos=pos,
                words=words or sum((t[0] for t in trees), []), hq=hq, hkv=hkv, preset=preset, n=n)


def run(env, p, max_tree=None, words=True, ws=True, expect=0, out=None, stream=None, n_rows=None, **score):
    kv, torch = env
    max_tree = max_tree or int(np.diff(p["cu"]).max())
    meta = kv.make_meta(p["hkv"], p["hq"], len(p["cache"]), max_blocks_per_seq=p["bt"].shape[1], preset=p["preset"])
    slopes = score.pop("slopes", None)
    out = torch.full((p["n"], p["hq"], 128), 7.0, dtype=torch.float16, device="cuda") if out is None else out
    scratch = torch.full((kv.tree_scratch_bytes(meta, len(p["lens"]), max_tree),), 255, dtype=torch.uint8, device="cuda")
    args = [to_dev(torch, p["q"]), to_dev(torch, p["k"]), to_dev(torch, p["v"]),
            words_to_dev(torch, p["words"]) if words else None, to_dev(torch, p["cu"]), to_dev(torch, p["lens"]), max_tree,
            to_dev(torch, p["bt"]), to_dev(torch, p["cache"]), to_dev(torch, p["ws"]) if ws else None, out, scratch, meta]
    torch.cuda.synchronize()
    kv.kvarn_tree_attention(*args, positions=to_dev(torch, p["pos"]), stream=stream,
                            slopes=None if slopes is None else to_dev(torch, np.asarray(slopes, np.float32)), **score)
    torch.cuda.synchronize()
    assert kv.kvarn_device_flags() == expect
    return out.view(torch.int16).cpu().numpy().view(np.float16).astype(np.float64)


def check(env, p, only=None, words=True, **kw):
    got = run(env, p, words=words, **kw)
    score = {x: kw[x] for x in ("scale", "softcap", "window", "slopes") if x in kw}
    want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"] if words else None, p["cu"], p["lens"], p["bt"], p["ws"],
                             p["cache"], positions=p["pos"], only=only, **score)
    rows = ~np.isnan(want)
    assert_decode_close(got[rows], want[rows])
    return got


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
def test_presets_ragged(env, preset):
    check(env, make([300, 128, 77, 0, 513], [5, 1, 8, 3, 2], 16, 2, preset))


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_groups(env, group):
    check(env, make([270, 129], [7, 3], 2 * group, 2, seed=71))


@pytest.mark.parametrize("t", [1, 2, 3, 4, 8, 9, 16, 17, 31, 33, 63, 64])
def test_tree_sizes(env, t):
    check(env, make([400], [t], 8, 1, seed=72))


@pytest.mark.parametrize("t", [1, 13, 64])
def test_chain_without_words(env, t):
    p = make([200, 5], [t, max(1, t // 2)], 10, 2, seed=73, chain=True)
    a = check(env, p, words=False)
    assert np.array_equal(a, run(env, p))


@pytest.mark.parametrize("lens", [[0], [1], [127], [128], [129], [255, 256], [1281], [0, 0, 0]])
def test_lengths(env, lens):
    check(env, make(lens, [4] * len(lens), 8, 2, seed=74))


@pytest.mark.parametrize("score", [
    dict(softcap=5.0), dict(softcap=30.0), dict(window=1), dict(window=2), dict(window=100), dict(window=128),
    dict(window=129), dict(window=100000), dict(slopes=[0.5, 0.25, 0.01, 0.0, 2.0, -0.01]), dict(scale=0.02),
    dict(scale=0.2, softcap=20.0, window=200, slopes=[0.5, 0.25, 0.01, 0.0, 2.0, -0.001]),
])
@pytest.mark.parametrize("preset", ["k4v2", "k2v2"])
def test_scores(env, score, preset):
    check(env, make([700, 130, 50, 256], [6, 3, 9, 1], 6, 2, preset, seed=75), **score)


def test_large_scores(env):
    """Scores of some hundreds: one key takes all the weight."""
    check(env, make([500, 300], [6, 3], 8, 1, seed=76, q_scale=40.0))
    check(env, make([500, 300], [6, 3], 8, 1, seed=76, q_scale=0.01))


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
def test_constant_and_biased_groups(env, preset):
    """Tiles whose groups are constant (keys equal over the tokens, values that rotate to a constant;
    their steps have the least value) or far from zero."""
    from oracle import kvarn_oracle as o
    rng = np.random.default_rng(92)
    p = make([900, 700], [5, 9], 8, 1, preset, seed=92)
    k, v = synth.prefill_kv(6 * 128, 1, seed=93)
    k, v = (x.reshape(6, 128, 128).copy() for x in (k, v))
    k[0] = k[0, :1]                                          # every token's key the same
    k[1] += np.float16(8) * rng.standard_normal(128).astype(np.float16)      # keys with a large mean
    v[2, ::3] = 0
    v[2, ::3, 0] = np.float16(1.5)                           # rotates to a constant
    v[3] = 0
    v[4, 5:90] += np.float16(6)                              # values with a large mean
    k[5], v[5] = np.float16(0.25), np.float16(0)
    p["cache"], _, _ = o.quantize_tiles(k[:, None], v[:, None], preset=preset)
    for bt in (p["bt"], np.where(p["bt"] >= 0, (p["bt"] + 1) % 6, p["bt"]).astype(np.int32)):
        p["bt"] = bt
        check(env, p)


def test_rows_that_attend_little(env):
    rng = np.random.default_rng(77)
    lens, counts = [0, 0, 140], [6, 64, 5]
    words = [0, 1, 2, 0, 63, 32] + [int(x) for x in rng.integers(0, 2 ** 63, 64)] + [0, 31, 16, 0, 1]
    words[6 + 5], words[6 + 6] = 1 << 63, (1 << 64) - 1
    p = make(lens, counts, 6, 2, seed=77, words=words)
    got = check(env, p)
    assert (got[[0, 3]] == 0).all()
    # a window that leaves nothing of the cache, with an empty word
    p["words"] = [0] * p["n"]
    p["pos"][:] = 100000
    got = check(env, p, window=5)
    assert (got == 0).all()


def test_zero_tokens_and_rows_of_no_sequence(env):
    p = make([300, 10, 200, 140], [3, 0, 4, 0], 8, 2, seed=78)
    p["cu"] = (p["cu"] + 2).astype(np.int32)
    for x in ("q", "k", "v"):
        p[x] = np.concatenate([p[x][:2], p[x], p[x][:3]])
    p["words"] = [1, 1] + p["words"] + [1, 1, 1]
    p["pos"] = np.concatenate([[0, 0], p["pos"], [0, 0, 0]]).astype(np.int32)
    p["n"] += 5
    got = check(env, p)
    assert (got[:2] == 7).all() and (got[9:] == 7).all()


def test_longer_than_max_tree(env):
    kv, _ = env
    p = make([200, 150], [7, 2], 8, 1, seed=79, chain=True)
    got = run(env, p, max_tree=4, expect=kv.FLAG_BAD_LENGTH)
    want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"], p["cu"], p["lens"], p["bt"], p["ws"], p["cache"])
    assert_decode_close(got[[0, 1, 2, 3, 7, 8]], want[[0, 1, 2, 3, 7, 8]])
    assert (got[4:7] == 7).all()
    # words of the first tokens that name the dropped ones
    p["words"] = [w | 0x7F for w in p["words"][:7]] + p["words"][7:]
    got = run(env, p, max_tree=4, expect=kv.FLAG_BAD_LENGTH)
    p["words"] = [w & 0xF for w in p["words"][:7]] + p["words"][7:]
    want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"], p["cu"], p["lens"], p["bt"], p["ws"], p["cache"])
    assert_decode_close(got[:4], want[:4])


def test_bad_blocks_and_lengths(env):
    kv, torch = env
    p = make([300, 300], [3, 2], 8, 2, seed=80)
    good = run(env, p)
    p["bt"] = p["bt"].copy()
    p["bt"][0, 1] = 99
    got = run(env, p, expect=kv.FLAG_BAD_BLOCK)
    assert np.isfinite(got).all() and np.array_equal(got[3:], good[3:])
    # the sequence as if the bad tile were not there: its other tile and its workspace
    q = make([172, 300], [3, 2], 8, 2, seed=80)
    q |= dict(bt=p["bt"], ws=p["ws"], cache=p["cache"])
    want = vo.tree_attention(q["q"], q["k"], q["v"], q["words"], q["cu"], q["lens"], q["bt"], q["ws"], q["cache"])
    assert_decode_close(got[:3], want[:3])
    # a table too short for the length; no workspace
    p = make([300], [3], 8, 1, seed=81)
    p["bt"] = p["bt"][:, :1].copy()
    got = run(env, p, expect=kv.FLAG_BAD_LENGTH)
    q = make([172], [3], 8, 1, seed=81) | dict(bt=p["bt"], ws=p["ws"])
    want = vo.tree_attention(q["q"], q["k"], q["v"], q["words"], q["cu"], q["lens"], q["bt"], q["ws"], q["cache"])
    assert_decode_close(got, want)
    got = run(env, p, ws=False, expect=kv.FLAG_BAD_LENGTH)
    q["lens"] = np.array([128], np.int32)
    want = vo.tree_attention(q["q"], q["k"], q["v"], q["words"], q["cu"], q["lens"], q["bt"], q["ws"], q["cache"])
    assert_decode_close(got, want)
    # a sequence whose rows end behind the tensors' is not computed
    p = make([300, 140], [3, 2], 8, 1, seed=82)
    p["cu"][2] += 1
    got = run(env, p, expect=kv.FLAG_BAD_LENGTH)
    assert (got[3:] == 7).all() and (got[:3] != 7).any()
    # a negative length is a length of 0
    p = make([0], [3], 8, 1, seed=83)
    want = run(env, p)
    p["lens"][:] = -300
    assert np.array_equal(run(env, p), want)


def test_many_sequences(env):
    rng = np.random.default_rng(84)
    lens = rng.integers(0, 600, 90).tolist()
    counts = rng.integers(0, 12, 90).tolist()
    check(env, make(lens, counts, 8, 2, seed=84))


def test_more_units_than_warps(env):
    rng = np.random.default_rng(85)
    lens = rng.integers(100, 300, 300).tolist()
    p = make(lens, [2] * 300, 8, 8, seed=85)
    check(env, p, only=[(int(s), int(h)) for s, h in zip(rng.integers(0, 300, 200), rng.integers(0, 8, 200))])


def test_long_context(env):
    """Long sequences, split over the whole GPU, at the sizes where shared blocks keep the oracle quick."""
    p = make([20000, 131072], [5, 8], 8, 1, seed=86)
    check(env, p)


def test_repeats_are_bit_equal(env):
    p = make([3000, 900, 77], [9, 4, 30], 16, 2, seed=87)
    a = run(env, p)
    for _ in range(3):
        assert np.array_equal(run(env, p), a)


def test_stream_and_graph(env):
    kv, torch = env
    p = make([1000, 200], [5, 9], 16, 2, seed=88)
    a = check(env, p, stream=torch.cuda.Stream())
    meta = kv.make_meta(2, 16, len(p["cache"]), max_blocks_per_seq=p["bt"].shape[1])
    outs = [torch.zeros(p["n"], 16, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
    scratch = torch.empty(kv.tree_scratch_bytes(meta, 2, 9), dtype=torch.uint8, device="cuda")
    args = [to_dev(torch, p["q"]), to_dev(torch, p["k"]), to_dev(torch, p["v"]), words_to_dev(torch, p["words"]),
            to_dev(torch, p["cu"]), to_dev(torch, p["lens"]), 9, to_dev(torch, p["bt"]), to_dev(torch, p["cache"]),
            to_dev(torch, p["ws"])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for out in outs:                         # two calls on one scratch, in order
            kv.kvarn_tree_attention(*args, out, scratch, meta)
    for _ in range(2):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert np.array_equal(out.view(torch.int16).cpu().numpy().view(np.float16).astype(np.float64), a)


def test_one_token_is_decode(env):
    """One new token over L tokens is the decode over L + 1 once that token is appended (no tile completed)."""
    kv, torch = env
    p = make([500, 130, 5], [1, 1, 1], 16, 2, seed=89)
    got = run(env, p)
    meta = kv.make_meta(2, 16, len(p["cache"]), max_blocks_per_seq=p["bt"].shape[1])
    ws, lens = to_dev(torch, p["ws"]), torch.zeros(3, dtype=torch.int32, device="cuda")
    cache, bt = to_dev(torch, p["cache"]), to_dev(torch, p["bt"])
    kv.kvarn_append_tokens(to_dev(torch, p["k"]), to_dev(torch, p["v"]), to_dev(torch, p["cu"]), to_dev(torch, p["lens"]),
                           lens, bt, ws, cache, meta)
    out = torch.empty(3, 16, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(kv.decode_scratch_bytes(meta, 3), dtype=torch.uint8, device="cuda")
    kv.kvarn_decode_attention(to_dev(torch, p["q"]), cache, ws, bt, lens, out, scratch, meta)
    want = out.float().cpu().numpy().astype(np.float64)
    ulp = np.spacing(np.abs(want).astype(np.float16)).astype(np.float64)
    assert (np.abs(got - want) <= 2 * 2e-3 + ulp).all()      # each within the decode tolerance


def test_verify_step_together(env):
    """Projected rows through norm and rotation, the tree, the accepted path's append (one
    sequence completes a tile) and the decode of the next token, all in one graph, twice over."""
    kv, torch = env
    hq, hkv, n_seqs, t = 16, 2, 3, 6
    lens = [300, 126, 255]
    cache0, bt, ws0 = paged("k4v2", lens, hkv, 90, width=4)
    for s, n in enumerate(lens):
        bt[s, n // 128] = 6 + s                           # the blocks that the step may complete
    cache0 = np.concatenate([cache0, np.zeros((3,) + cache0.shape[1:], np.uint8)])
    rng = np.random.default_rng(90)
    words, depths = zip(*[random_tree(t, rng) for _ in range(n_seqs)])
    pos = np.array([lens[s] + d for s in range(n_seqs) for d in depths[s]], np.int32)
    acc = np.array([[0, 2, 4], [1, 3, 5], [0, 1, 2]], np.int32)
    n_acc = np.array([2, 3, 0], np.int32)
    cu = np.arange(n_seqs + 1, dtype=np.int32) * t
    qkv = (torch.randn(n_seqs * t, (hq + 2 * hkv) * 128, device="cuda",
                       generator=torch.Generator(device="cuda").manual_seed(90)) * 2).bfloat16()
    inv = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    meta = kv.make_meta(hkv, hq, len(cache0), max_blocks_per_seq=4)
    d = {x: to_dev(torch, y) for x, y in dict(bt=bt, lens=np.array(lens, np.int32), pos=pos, acc=acc, n_acc=n_acc, cu=cu,
                                              cache=cache0, ws=ws0).items()}
    d["words"] = words_to_dev(torch, sum(map(list, words), []))
    q, k, v = (torch.empty(n_seqs * t, h, 128, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv))
    out, nxt = torch.empty_like(q), torch.empty(n_seqs, hq, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(max(kv.tree_scratch_bytes(meta, n_seqs, t), kv.decode_scratch_bytes(meta, n_seqs)),
                          dtype=torch.uint8, device="cuda")
    lens1 = torch.zeros_like(d["lens"])
    parts = [x.unflatten(1, (-1, 128)) for x in qkv.split([hq * 128, hkv * 128, hkv * 128], 1)]

    def step():
        kv.kvarn_qk_norm_rope(*parts, d["pos"], q, k, v, meta, q_weight=w, k_weight=w, inv_freq=inv)
        kv.kvarn_tree_attention(q, k, v, d["words"], d["cu"], d["lens"], t, d["bt"], d["cache"], d["ws"], out, scratch, meta)
        kv.kvarn_append_tokens(k, v, d["cu"], d["lens"], lens1, d["bt"], d["ws"], d["cache"], meta, accepted=d["acc"],
                               n_accepted=d["n_acc"])
        kv.kvarn_decode_attention(q[:n_seqs], d["cache"], d["ws"], d["bt"], lens1, nxt, scratch, meta)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        d["cache"].copy_(to_dev(torch, cache0))
        d["ws"].copy_(to_dev(torch, ws0))
        for x in (q, k, v, out, nxt, lens1):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert kv.kvarn_device_flags() == 0
        f = {x: y.view(torch.int16).cpu().numpy().view(np.float16) for x, y in dict(q=q, k=k, v=v).items()}
        raw = parts[0].double().cpu().numpy()
        ref = vo.qk_norm_rope(raw, np.ones(128), 1e-6, inv.cpu().numpy(), pos, False)
        assert np.abs(f["q"] - ref).max() <= 2.0 ** -10 * np.abs(ref).max()
        want = vo.tree_attention(f["q"], f["k"], f["v"], sum(map(list, words), []), cu, lens, bt, ws0, cache0)
        assert_decode_close(out.float().cpu().numpy(), want)
        ws1, _, l1, done = vo.append_tokens(f["k"], f["v"], cu, lens, bt, ws0, cache0, accepted=acc, n_accepted=n_acc)
        assert np.array_equal(lens1.cpu().numpy(), l1) and [x[0] for x in done] == [1]
        assert np.array_equal(d["ws"].view(torch.int16).cpu().numpy().view(np.float16), ws1)
        from oracle import kvarn_oracle as o
        want = o.decode(f["q"][:n_seqs].astype(np.float64), d["cache"].cpu().numpy(), ws1, bt, l1)
        assert_decode_close(nxt.float().cpu().numpy(), want)


@pytest.mark.parametrize("hq,counts", [(16, [5, 1, 16]), (64, [7, 13, 2])])
@pytest.mark.parametrize("place", ["value", "key", "query", "workspace"])
def test_infinities_stay_with_the_rows_that_attend_them(env, hq, counts, place):
    """Infinities and NaN in a drafted token's value or key, in a query row, and in a workspace token
    that a window leaves out: rows that attend them become what the definition says, the others
    are as if they were not there."""
    score = dict(window=200) if place == "workspace" else {}
    p = make([300, 70, 257], counts, hq, 8, seed=130)
    cu = p["cu"]
    if place == "value":
        p["v"][cu[0] + 2, 3, [5, 6, 127]] = np.float16([np.inf, np.nan, -np.inf])
        p["v"][cu[2], 0, 64] = -np.inf
    elif place == "key":
        p["k"][cu[0] + 1, 2, 17] = np.nan
        p["k"][cu[2] + 1, 7, 0] = np.inf
    elif place == "query":
        p["q"][cu[0] + 1, 3, 9] = np.inf
        p["q"][cu[2], hq - 1, 100] = np.nan
    else:
        p["pos"][:] = np.where(np.arange(p["n"]) % 2 == 0, 600, 400)      # windows from 401 on, and from 201 on
        p["ws"][0, 1, 1, 20, 3] = np.nan                                   # position 276
        p["ws"][2, 4, 1, 0, 8] = np.inf                                    # position 256
    got = run(env, p, **score)
    with np.errstate(all="ignore"):
        want = vo.tree_attention(p["q"], p["k"], p["v"], p["words"], p["cu"], p["lens"], p["bt"], p["ws"], p["cache"],
                                 positions=p["pos"], **score)
    bad = ~np.isfinite(want)
    assert bad.any() and not bad.all()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
    assert_decode_close(got[~bad], want[~bad])
