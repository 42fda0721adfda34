"""Rotation along several axes, decode attention that weighs its tiles, and eviction on the GPU,
against their float64 definitions."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import budget_ops as bo
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.verify_common import TINY, paged, record_pool, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import kv_cache_quantization_x128_gb300 as kv
    torch.cuda.set_device(0)
    kv.kvarn_device_flags()
    return kv, torch


# ------------------------------------------------------------------ rotation along several axes
def _axes_check(env, n, hq, hkv, dtype, sections, mixed=False, interleaved=False, norm=True, with_v=True, far=3000,
                expanded=False, in_place=False, stream=None):
    kv, torch = env
    g = torch.Generator().manual_seed(n * 37 + hq)
    t = getattr(torch, dtype)
    axes = [a for a, c in enumerate(sections) for _ in range(c)]
    if mixed:
        axes = [axes[(7 * i) % len(axes)] for i in range(len(axes))]
    half, na = len(axes), len(sections)
    x = (torch.randn(n, (hq + 2 * hkv) * 128 + 64, generator=g) * 3).to(t).cuda()
    q, k, v = (p.unflatten(1, (-1, 128)) for p in x[:, :-64].split([hq * 128, hkv * 128, hkv * 128], 1))
    if in_place:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = ((1 + 0.3 * torch.randn(128, generator=g)).to(t).cuda() if norm else None for _ in range(2))
    pos = torch.randint(0, far, (na, n), generator=g, dtype=torch.int32)
    if expanded:
        pos = pos[:1].expand(na, n)
    inv = (1e4 ** (-torch.arange(half) / half)).float()
    # rows of a wider array, each axis at a stride of its own
    held = pos[:1].cuda().expand(na, n) if expanded else torch.zeros(na, n + 12, dtype=torch.int32, device="cuda")
    if not expanded:
        held[:, :n] = pos.cuda()
        held = held[:, :n]
    want, plain = [], []
    for p, w in ((q, qw), (k, kw)):
        a = p.cpu().double().numpy()
        ww = None if w is None else w.cpu().double().numpy()
        want.append(bo.qk_norm_rope_axes(a, ww, 1e-6, inv.numpy(), pos.numpy(), axes, interleaved))
        plain.append(vo.qk_norm_rope(a, ww, 1e-6, None, None, False))
    want.append(v.cpu().double().numpy())
    plain.append(want[2])
    outs = [q, k, v] if in_place else [torch.full((n, h, 128), 7.0, dtype=torch.float16, device="cuda")
                                       for h in (hq, hkv, hkv)]
    torch.cuda.synchronize()
    kv.kvarn_qk_norm_rope_axes(q, k, v if with_v else None, held, axes, outs[0], outs[1], outs[2] if with_v else None,
                               kv.make_meta(hkv, hq, 1, 1), q_weight=qw, k_weight=kw, inv_freq=inv.cuda(),
                               interleaved=interleaved, stream=stream)
    torch.cuda.synchronize()
    if not with_v:
        assert bool((outs[2] == 7).all())
    for out, ref, raw in list(zip(outs, want, plain))[: 3 if with_v else 2]:
        # (counted as in tests/test_verify_gpu.py: the arithmetic is the same)
        tol = 2.0 ** -11 * np.abs(ref) + TINY["float16"] + 2.0 ** -19 * 2 * np.abs(raw).max(-1, keepdims=True)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sections,mixed", [((16, 24, 24), False), ((24, 20, 20), True), ((32, 32), False), ((3, 5), True),
                                            ((10, 18, 20, 16), True), ((64,), False), ((0, 8, 24), False)])
def test_axes_types(env, dtype, interleaved, sections, mixed):
    _axes_check(env, 7, 5, 1, dtype, sections, mixed, interleaved)


@pytest.mark.parametrize("n,hq,hkv", [(1, 64, 8), (1, 1, 1), (37, 28, 4), (303, 40, 8), (2501, 16, 2)])
def test_axes_sizes(env, n, hq, hkv):
    _axes_check(env, n, hq, hkv, "bfloat16", (16, 24, 24))


def test_axes_without_parts_and_in_place(env):
    kv, torch = env
    _axes_check(env, 9, 8, 2, "float16", (16, 16), norm=False)
    _axes_check(env, 9, 8, 2, "float32", (16, 24, 24), with_v=False)
    _axes_check(env, 40, 8, 2, "float16", (16, 24, 24), in_place=True)
    _axes_check(env, 9, 8, 2, "float16", (16, 24, 24), expanded=True)
    _axes_check(env, 6, 2, 1, "float16", (16, 24, 24), far=2 ** 31 - 1)
    _axes_check(env, 33, 8, 2, "float16", (16, 24, 24), stream=torch.cuda.Stream())


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_text_is_rotated_as_by_one_axis(env, dtype):
    kv, torch = env
    q, k, v = (torch.randn(50, h, 128, device="cuda").to(getattr(torch, dtype)) for h in (8, 2, 2))
    pos = torch.randint(0, 1 << 20, (50,), device="cuda", dtype=torch.int32)
    inv = (1e6 ** (-torch.arange(64, device="cuda") / 64)).float()
    w = 1 + torch.randn(128, device="cuda").to(q.dtype) / 4
    a, b = ([torch.empty(50, h, 128, dtype=torch.float16, device="cuda") for h in (8, 2, 2)] for _ in range(2))
    meta = kv.make_meta(2, 8, 1, 1)
    kv.kvarn_qk_norm_rope(q, k, v, pos, *a, meta, q_weight=w, k_weight=w, inv_freq=inv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kvarn_qk_norm_rope_axes(q, k, v, pos.expand(3, 50), [i % 3 for i in range(64)], *b, meta, q_weight=w, k_weight=w,
                                   inv_freq=inv)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


# ------------------------------------------------------------------ attention that weighs its tiles
def _weigh(env, p, decay=1.0, expect=0, lse=True, stream=None):
    """The call over numpy inputs; (out, lse, weights) as float64."""
    kv, torch = env
    n, hq, _ = p["q"].shape
    hkv = p["cache"].shape[1]
    meta = kv.make_meta(hkv, hq, p["cache"].shape[0], p["bt"].shape[1], preset=p["preset"])
    d = {x: None if p[x] is None else to_dev(torch, p[x]) for x in ("q", "cache", "ws", "bt", "lens", "w")}
    out = torch.full((n, hq, 128), float("nan"), dtype=torch.float16, device="cuda")
    ls = torch.full((n, hq), float("nan"), device="cuda") if lse else None
    scratch = torch.randint(0, 256, (kv.decode_weights_scratch_bytes(meta, n),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    kv.kvarn_decode_attention_weights(d["q"], d["cache"], d["ws"], d["bt"], d["lens"], d["w"], out, scratch, meta,
                                      decay=decay, lse=ls, stream=stream)
    torch.cuda.synchronize()
    assert kv.kvarn_device_flags() == expect
    return (out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None, d["w"].double().cpu().numpy())


def _make(lens, hq, hkv, preset="k4v2", seed=1, width=None):
    lens = np.asarray(lens, np.int32)
    cache, bt, ws = paged(preset, lens, hkv, seed, width=width)
    w = np.random.default_rng(seed).exponential(0.1, (len(lens), hkv, bt.shape[1])).astype(np.float32)
    return dict(q=synth.queries(len(lens), hq, seed), cache=cache, bt=bt, ws=ws, lens=lens, w=w, preset=preset)


def _weigh_check(env, p, decay=1.0, got=None, pairs=None):
    out, lse, w = got or _weigh(env, p, decay)
    hkv = p["cache"].shape[1]
    want, lse_want, w_want = bo.decode_weights(p["q"], p["cache"], p["ws"], p["bt"], p["lens"], p["w"], decay)
    assert_decode_close(out, want)
    g = p["q"].shape[1] // hkv
    for s in range(len(p["lens"])):
        t = -(-max(int(p["lens"][s]), 0) // 128)
        assert np.array_equal(w[s, :, t:], p["w"][s, :, t:].astype(np.float64))
        if t == 0:
            assert (lse[s] == -np.inf).all()
            continue
        for h in range(hkv):
            eps = bo.score_error(p["q"], p["cache"], p["ws"], p["bt"], p["lens"], s, h, p["preset"])
            # a sum of exponentials: scores off by eps, 2 ulp of each exponential, below 64 roundings
            ref = lse_want[s, h * g:(h + 1) * g]
            assert (np.abs(lse[s, h * g:(h + 1) * g] - ref) <= eps + 2.0 ** -17 + 2.0 ** -22 * np.abs(ref)).all()
            ref = w_want[s, h, :t]
            mass = ref - decay * p["w"][s, h, :t].astype(np.float64)
            tol = mass * (2 * eps + 2.0 ** -15) + 2.0 ** -22 * ref + 1e-37
            err = np.abs(w[s, h, :t] - ref)
            assert (err <= tol).all(), (s, h, (err / tol).max())


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("hq,hkv", [(8, 1), (6, 2), (5, 1), (2, 2)])
def test_weigh_lengths(env, preset, hq, hkv):
    _weigh_check(env, _make([1, 127, 128, 129, 0, 255, 256, 1000, 2049, 17], hq, hkv, preset, seed=hq))


@pytest.mark.parametrize("decay", [0.0, 0.5, 0.999])
def test_weigh_fades(env, decay):
    p = _make([500, 128, 3, 900], 8, 2, seed=7)
    if decay == 0:
        p["w"][:, :, :1] = np.nan                  # what is replaced is not looked at
        got = _weigh(env, p, 0.0)
        p["w"][:, :, :1] = 0
        _weigh_check(env, p, 0.0, got)
    else:
        _weigh_check(env, p, decay)


@pytest.mark.parametrize("preset", ["k4v2", "k2v2"])
def test_weigh_many_units_and_one_long(env, preset):
    """Both shapes of the split: more units than SMs, and one sequence cut over all of them."""
    rng = np.random.default_rng(3)
    _weigh_check(env, _make(rng.integers(0, 700, 90), 4, 2, preset, seed=11))
    _weigh_check(env, _make([40000], 8, 1, preset, seed=12))


def test_weigh_is_the_decode_and_the_same_each_time(env):
    kv, torch = env
    p = _make([3000, 128 * 9, 5, 0, 777], 16, 2, seed=13)
    a, b = _weigh(env, p, 0.9), _weigh(env, p, 0.9)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))
    assert np.array_equal(_weigh(env, p, 0.9, lse=False)[2], a[2])
    meta = kv.make_meta(2, 16, p["cache"].shape[0], p["bt"].shape[1])
    out = torch.empty(5, 16, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(kv.decode_scratch_bytes(meta, 5), dtype=torch.uint8, device="cuda")
    d = {x: to_dev(torch, p[x]) for x in ("q", "cache", "ws", "bt", "lens")}
    kv.kvarn_decode_attention(d["q"], d["cache"], d["ws"], d["bt"], d["lens"], out, scratch, meta)
    assert np.abs(out.double().cpu().numpy() - a[0]).max() <= 4e-3 + 2.0 ** -9 * np.abs(a[0]).max()


def test_weigh_data_errors(env):
    kv, _ = env
    # a block that is not there: its tile gets nothing, the others share the weight
    p = _make([700, 300], 8, 2, seed=14)
    p["bt"][0, 2] = 99
    out, lse, w = _weigh(env, p, 0.5, expect=kv.FLAG_BAD_BLOCK)
    assert np.array_equal(w[0, :, 2], 0.5 * p["w"][0, :, 2].astype(np.float64))
    new = w - 0.5 * p["w"]
    assert np.allclose(new[0, :, :6].sum(1), 4, atol=1e-4) and np.isfinite(out).all()
    # no block there at all
    p = _make([256], 8, 2, seed=15)
    p["bt"][:] = -1
    out, lse, w = _weigh(env, p, expect=kv.FLAG_BAD_BLOCK)
    assert (out == 0).all() and (lse == -np.inf).all() and np.array_equal(w, p["w"].astype(np.float64))
    # without a workspace
    p = _make([300], 8, 2, seed=16)
    q = dict(p, ws=None)
    out, lse, w = _weigh(env, q, expect=kv.FLAG_BAD_LENGTH)
    assert np.array_equal(w[:, :, 2:], p["w"][:, :, 2:].astype(np.float64))
    whole = dict(p, lens=np.array([256], np.int32))
    _weigh_check(env, whole, got=(out, lse, w))
    # longer than its table: the tiles of the table and the workspace tokens, whose weight has no entry
    p = _make([5 * 128 + 60], 4, 1, seed=17)
    full = p["bt"]
    p["bt"], p["w"] = full[:, :2].copy(), p["w"][:, :, :2].copy()
    out, lse, w = _weigh(env, p, expect=kv.FLAG_BAD_LENGTH)
    k, v = vo.cached_tokens(p["cache"], p["ws"], full[0], 0, 700, 0)
    mine = np.concatenate([np.arange(256), np.arange(640, 700)])
    x = p["q"][0].astype(np.float64) @ k[mine].T / np.sqrt(128)
    e = np.exp(x - x.max(1, keepdims=True))
    e /= e.sum(1, keepdims=True)
    assert_decode_close(out, (e @ v[mine])[None])
    assert np.allclose(w[0, 0] - p["w"][0, 0], [e[:, :128].sum(), e[:, 128:256].sum()], atol=1e-4)
    # a table that ends with the last whole tile: the partial tile's weight is dropped
    p = _make([300], 8, 2, seed=18, width=2)
    _weigh_check(env, p)


def test_weigh_without_blocks(env):
    kv, torch = env
    ws = synth.workspace_tokens(2, 1, seed=5)
    q, lens = synth.queries(2, 4, 5), np.array([50, 0], np.int32)
    meta = kv.make_meta(1, 4, 0, 0)
    out = torch.empty(2, 4, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(kv.decode_weights_scratch_bytes(meta, 2), dtype=torch.uint8, device="cuda")
    kv.kvarn_decode_attention_weights(to_dev(torch, q), None, to_dev(torch, ws), None, to_dev(torch, lens), None, out,
                                      scratch, meta)
    assert kv.kvarn_device_flags() == 0
    want = o.attend(q[0].astype(np.float64), ws[0, 0, 0, :50].astype(np.float64), ws[0, 0, 1, :50].astype(np.float64))
    assert_decode_close(out.double().cpu().numpy(), np.stack([want, np.zeros((4, 128))]))


def _quantized(k, v, preset):
    """Tiles [n, tokens, 128] of one kv-head as a cache of n blocks."""
    return o.quantize_tiles(np.asarray(k, np.float16)[:, None], np.asarray(v, np.float16)[:, None], preset=preset)[0]


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("k_mean,k_std,v_mean,v_std", [(0, 1, 1, 0.3), (3, 0.3, 0, 1), (-30, 0.5, 200, 0.5),
                                                       (0, 3e-4, 0, 3e-4)])
def test_weigh_tensors_of_any_scale(env, preset, k_mean, k_std, v_mean, v_std):
    """Means of several times the spread drive the normalisation's scales far apart: r s to 2^-19, c s beyond fp16."""
    rng = np.random.default_rng(21)
    p = _make([3 * 128 + 40], 8, 1, preset, seed=21)
    k, v = rng.normal(k_mean, k_std, (3, 128, 128)), rng.normal(v_mean, v_std, (3, 128, 128))
    p["cache"], p["bt"] = _quantized(k, v, preset), np.array([[0, 1, 2, -1]], np.int32)
    p["ws"][0, 0, 0], p["ws"][0, 0, 1] = rng.normal(k_mean, k_std, (128, 128)), rng.normal(v_mean, v_std, (128, 128))
    _weigh_check(env, p)


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2"])
@pytest.mark.parametrize("where", ["tile", "workspace", "other"])
def test_weigh_values_a_million_times_apart(env, preset, where):
    """Behind a token that takes nearly all the weight with a value of 0.01: tokens of 10^-5 of it with values of 10^4."""
    rng = np.random.default_rng(22)
    n = 128 + 60
    k, v = 0.01 * rng.standard_normal((n, 128)), 1e4 * rng.standard_normal((n, 128))
    sink = {"tile": 5, "workspace": 140, "other": 140}[where]
    k[sink], v[sink] = 0, 0.01
    k[sink, 7] = 13.0
    if where == "other":
        v[128:] = 0.01
    if where == "workspace":
        v[:128] = 0.01
    p = _make([n], 8, 1, preset, seed=22)
    p["cache"], p["bt"] = _quantized(k[None, :128], v[None, :128], preset), np.array([[0, -1]], np.int32)
    p["ws"][0, 0, 0, :60], p["ws"][0, 0, 1, :60] = k[128:], v[128:]
    q = 0.01 * rng.standard_normal((1, 8, 128))
    q[..., 7] = 10 + np.arange(8) / 8
    p["q"] = q.astype(np.float16)
    _weigh_check(env, p)


@pytest.mark.parametrize("preset", ["k4v2", "k2v2"])
def test_weigh_scores_far_out(env, preset):
    """Scores of 10^8 and more: one token takes all of a row's weight."""
    rng = np.random.default_rng(23)
    p = _make([256 + 40], 8, 1, preset, seed=23)
    k = (2e4 * rng.standard_normal((2, 128, 128))).clip(-6e4, 6e4)
    p["cache"], p["bt"] = _quantized(k, rng.standard_normal((2, 128, 128)), preset), np.array([[0, 1, -1]], np.int32)
    p["ws"][0, 0, 0, :40] = (2e4 * rng.standard_normal((40, 128))).clip(-6e4, 6e4)
    p["q"] = (5e4 / 3 * np.clip(rng.standard_normal((1, 8, 128)), -3, 3)).astype(np.float16)
    out, lse, w = _weigh(env, p)
    want, lse_want, w_want = bo.decode_weights(p["q"], p["cache"], p["ws"], p["bt"], p["lens"], p["w"])
    assert_decode_close(out, want)
    assert np.allclose(w, w_want, atol=1e-4) and np.allclose(lse, lse_want, rtol=1e-5)


def test_weigh_what_is_not_finite_stays_in_its_sequence(env):
    p = _make([300, 300, 200], 8, 2, seed=24)
    clean = _weigh(env, p)
    p["q"][1, 3] = np.nan
    p["ws"][2, 1, 1, 60] = np.inf                  # an attended value
    p["ws"][0, 0, :, 100:] = np.nan                # rows behind the sequence's last token
    out, lse, w = _weigh(env, p)
    assert np.array_equal(out[0], clean[0][0]) and np.array_equal(w[0], clean[2][0])
    assert np.isnan(out[1, 3]).all() and np.array_equal(out[1, :3], clean[0][1, :3])
    assert np.array_equal(out[1, 4:], clean[0][1, 4:]) and np.array_equal(w[1, 1], clean[2][1, 1])
    assert np.array_equal(out[2, :4], clean[0][2, :4]) and not np.isfinite(out[2, 4:]).any()
    assert np.array_equal(w[2], clean[2][2])


def test_weigh_stream_and_graph(env):
    kv, torch = env
    p = _make([700, 129, 0, 4000], 8, 2, seed=25)
    once = _weigh(env, p, 0.75, stream=torch.cuda.Stream())
    meta = kv.make_meta(2, 8, p["cache"].shape[0], p["bt"].shape[1])
    d = {x: to_dev(torch, p[x]) for x in ("q", "cache", "ws", "bt", "lens", "w")}
    out = torch.empty(4, 8, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(kv.decode_weights_scratch_bytes(meta, 4), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kvarn_decode_attention_weights(d["q"], d["cache"], d["ws"], d["bt"], d["lens"], d["w"], out, scratch, meta,
                                          decay=0.75)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), once[0])
    assert np.array_equal(d["w"].double().cpu().numpy(), once[2])
    graph.replay()                                 # the weights go on from what the first replay left
    torch.cuda.synchronize()
    again = _weigh(env, dict(p, w=once[2].astype(np.float32)), 0.75)
    assert np.array_equal(d["w"].double().cpu().numpy(), again[2])


# ------------------------------------------------------------------ eviction
def _evict(env, w, lens, bt, budgets, cache, first, last, preset="k2v2", expect=0, in_place=False, stream=None):
    kv, torch = env
    hkv = cache.shape[1]
    meta = kv.make_meta(hkv, hkv, cache.shape[0], bt.shape[1], preset=preset)
    assert kv.meta_record_bytes(meta) == cache.shape[2]
    lens, budgets = np.asarray(lens, np.int32), np.asarray(budgets, np.int32)
    d = [to_dev(torch, x) for x in (w, lens, bt, budgets, cache)]
    wo = d[0] if in_place else torch.full_like(d[0], 7.0)
    kept, lo = torch.full(w.shape, 77, dtype=torch.int32, device="cuda"), torch.full_like(d[1], -5)
    torch.cuda.synchronize()
    kv.kvarn_evict_tiles(d[0], wo, d[1], lo, d[2], d[3], kept, d[4], meta, keep_first=first, keep_last=last, stream=stream)
    torch.cuda.synchronize()
    assert kv.kvarn_device_flags() == expect
    got = [x.cpu().numpy() for x in (kept, lo, wo, d[4])]
    want = bo.evict_tiles(w, lens, bt, budgets, cache, first, last)
    for name, a, b in zip(("kept", "lengths", "weights", "cache"), got, want):
        assert np.array_equal(a, b, equal_nan=name == "weights"), name
    return got


def _tiles(tiles, hkv, preset="k2v2", seed=1, tail=5, spare=2, width=None):
    """Records of random bytes (eviction does not look into them), blocks in a random order."""
    rng = np.random.default_rng(seed)
    lens = np.asarray([t * 128 + tail for t in tiles], np.int32)
    width = width or max(tiles) + 1
    used = [min(t + (tail > 0), width) for t in tiles]
    perm = rng.permutation(sum(used) + spare)
    bt, at = np.full((len(tiles), width), -1, np.int32), 0
    for s, u in enumerate(used):
        bt[s, :u] = perm[at:at + u]
        at += u
    cache = rng.integers(0, 256, (len(perm), hkv, o.LAYOUTS[preset].record_bytes), dtype=np.uint8)
    w = rng.lognormal(0, 2, (len(tiles), hkv, width)).astype(np.float32)
    w[rng.random(w.shape) < 0.1] = 0
    return w, lens, bt, cache


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("first,last", [(0, 0), (1, 2), (4, 1), (3, 50)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_choices(env, preset, first, last, in_place):
    w, lens, bt, cache = _tiles([13, 0, 1, 40, 7, 33, 12], 2, preset, seed=first + last)
    _evict(env, w, lens, bt, [6, 0, 0, 39, 7, 9, 100], cache, first, last, preset, in_place=in_place)


@pytest.mark.parametrize("tiles,hkv,keep", [([31, 32, 33, 64, 65], 3, 20), ([300], 1, 123), ([300, 257, 256], 2, 299),
                                            ([1100], 2, 400), ([2500, 90], 1, 64), ([9000], 1, 8000)])
@pytest.mark.parametrize("tail", [0, 127])
def test_evict_sizes(env, tiles, hkv, keep, tail):
    """Blocks of one warp and of many, several tiles a thread."""
    w, lens, bt, cache = _tiles(tiles, hkv, seed=len(tiles), tail=tail)
    _evict(env, w, lens, bt, [keep] * len(tiles), cache, 1, 2)


def test_evict_more_tiles_than_keys_are_held(env):
    w, lens, bt, cache = _tiles([12000], 1, seed=31)
    _evict(env, w, lens, bt, [11990], cache, 2, 3, in_place=True)
    _evict(env, w, lens, bt, [5000], cache, 0, 0)


def test_evict_ties_and_what_is_no_number(env):
    for seed in range(4):
        w, lens, bt, cache = _tiles([50, 200, 900], 2, seed=40 + seed)
        w[:] = np.random.default_rng(seed).integers(0, 3, w.shape)
        _evict(env, w, lens, bt, [20, 77, 300], cache, 1, 1, in_place=seed % 2 == 1)
        w[:, 0] = 0
        w[:, 1] = -np.float32(0)
        _evict(env, w, lens, bt, [20, 77, 300], cache, 0, 0)
        w[..., ::3] = np.nan
        w[..., 1::7] = np.inf
        w[..., 2::5] = -np.inf
        w[..., 3::11] = -1.5
        w[..., 5::13] = 1e-42
        _evict(env, w, lens, bt, [10, 160, 800], cache, 1, 4)


def test_evict_budgets_at_the_ends(env):
    w, lens, bt, cache = _tiles([9] * 7, 2, seed=50)
    _evict(env, w, lens, bt, [-1, 0, 1, 2, 8, 9, 2 ** 31 - 1], cache, 1, 2)
    _evict(env, w, lens, bt, [-2 ** 31, 0, 1, 2, 3, 4, 5], cache, 2 ** 31 - 1, 2 ** 31 - 1)
    lens[:3] = [-7, 0, 127]
    _evict(env, w, lens, bt, [3] * 7, cache, 1, 2)


def test_evict_data_errors_leave_the_sequence(env):
    kv, _ = env
    w, lens, bt, cache = _tiles([9, 9, 9], 2, seed=51)
    bt[1, 4] = len(cache)
    _evict(env, w, lens, bt, [5, 5, 5], cache, 1, 2, expect=kv.FLAG_BAD_BLOCK)
    _evict(env, w, lens, bt, [5, 9, 5], cache, 1, 2)                     # nothing to evict: not looked at
    bt[1, 4] = -1
    _evict(env, w, lens, bt, [5, 5, 5], cache, 1, 2, expect=kv.FLAG_BAD_BLOCK, in_place=True)
    bt[1, 4] = 0
    w, lens, bt, cache = _tiles([9, 9, 9], 2, seed=52)
    lens[2] = 128 * 10 + 128
    _evict(env, w, lens, bt, [5, 5, 5], cache, 1, 2, expect=kv.FLAG_BAD_LENGTH)


def test_evict_shared_prompts_stay_shared(env):
    """Two sequences with the same first two blocks, which stay in place for both."""
    w, lens, bt, cache = _tiles([20, 20], 2, seed=53)
    bt[1, :2] = bt[0, :2]
    before = cache[bt[0, :2]].copy()
    got = _evict(env, w, lens, bt, [8, 11], cache, 2, 1)
    assert np.array_equal(got[3][bt[0, :2]], before)


def test_evict_stream_and_graph(env):
    kv, torch = env
    _evict(env, *_first4(_tiles([60, 41], 4, seed=54), [20, 30]), 1, 2, stream=torch.cuda.Stream())
    w, lens, bt, cache = _tiles([60, 41], 4, seed=55)
    meta = kv.make_meta(4, 4, cache.shape[0], bt.shape[1], preset="k2v2")
    budgets = np.array([20, 30], np.int32)
    d = [to_dev(torch, x) for x in (w, lens, bt, budgets, cache)]
    wo, lo, kept = torch.empty_like(d[0]), torch.empty_like(d[1]), torch.empty(w.shape, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kvarn_evict_tiles(d[0], wo, d[1], lo, d[2], d[3], kept, d[4], meta, keep_first=1, keep_last=2)
    graph.replay()
    torch.cuda.synchronize()
    want = bo.evict_tiles(w, lens, bt, budgets, cache, 1, 2)
    for a, b in zip((kept, lo, wo, d[4]), want):
        assert np.array_equal(a.cpu().numpy(), b)


def _first4(t, budgets):
    w, lens, bt, cache = t
    return w, lens, bt, budgets, cache


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("preset", ["k4v2", "k4v4"])
def test_a_serving_loop_within_a_budget(env, preset):
    """Tokens of a video are rotated, appended, attended with weights; sequences above their budget lose tiles. Each step's
    output, weights and choice are checked against the definitions over the cache's own records."""
    kv, torch = env
    hq, hkv, n, width = 8, 2, 3, 8
    rng = np.random.default_rng(60)
    lens = np.array([6 * 128 + 126, 5 * 128 + 125, 3 * 128 + 127], np.int32)
    pool = record_pool(preset, 6, hkv, 0)
    cache = np.concatenate([pool, pool, pool, pool])                     # 24 blocks, a sequence's own 8
    bt = np.arange(n * width, dtype=np.int32).reshape(n, width)
    ws = synth.workspace_tokens(n, hkv, seed=61)
    meta = kv.make_meta(hkv, hq, len(cache), width, preset=preset)
    d_cache, d_ws, d_bt = to_dev(torch, cache), to_dev(torch, ws), to_dev(torch, bt)
    d_lens = [to_dev(torch, lens), torch.empty(n, dtype=torch.int32, device="cuda")]
    weights = torch.zeros(n, hkv, width, device="cuda")
    kept = torch.empty(n, hkv, width, dtype=torch.int32, device="cuda")
    budgets = torch.tensor([5, 5, 4], dtype=torch.int32, device="cuda")
    inv = (1e6 ** (-torch.arange(64, device="cuda") / 64)).float()
    axes = [0] * 16 + [1] * 24 + [2] * 24
    scratch = torch.empty(kv.decode_weights_scratch_bytes(meta, n), dtype=torch.uint8, device="cuda")
    q, k, v, out = (torch.empty(n, h, 128, dtype=torch.float16, device="cuda") for h in (hq, hkv, hkv, hq))
    for step in range(6):
        x = torch.tensor(rng.standard_normal((n, hq + 2 * hkv, 128)), dtype=torch.bfloat16).cuda()
        pos = torch.tensor(rng.integers(0, 3000, (3, n)), dtype=torch.int32).cuda()
        kv.kvarn_qk_norm_rope_axes(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, axes, q, k, v, meta, inv_freq=inv)
        kv.kvarn_append_decode(k, v, d_lens[0], d_lens[1], d_bt, d_ws, d_cache, meta)
        before = weights.cpu().numpy()
        kv.kvarn_decode_attention_weights(q, d_cache, d_ws, d_bt, d_lens[1], weights, out, scratch, meta, decay=0.9)
        torch.cuda.synchronize()
        c, w_s, ln = d_cache.cpu().numpy(), d_ws.cpu().numpy(), d_lens[1].cpu().numpy()
        p = dict(q=q.cpu().numpy(), cache=c, ws=w_s, bt=bt, lens=ln, w=before, preset=preset)
        lse = bo.decode_weights(p["q"], c, w_s, bt, ln, before, 0.9)[1]
        _weigh_check(env, p, 0.9, got=(out.double().cpu().numpy(), lse, weights.double().cpu().numpy()))
        held = weights.cpu().numpy()
        kv.kvarn_evict_tiles(weights, weights, d_lens[1], d_lens[0], d_bt, budgets, kept, d_cache, meta, keep_first=1,
                             keep_last=1)
        torch.cuda.synchronize()
        want = bo.evict_tiles(held, ln, bt, budgets.cpu().numpy(), c, 1, 1)
        for a, b in zip((kept, d_lens[0], weights, d_cache), want):
            assert np.array_equal(a.cpu().numpy(), b)
        assert kv.kvarn_device_flags() == 0
    assert (d_lens[0].cpu().numpy() // 128 <= [5, 5, 4]).all()
