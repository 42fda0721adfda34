"""The calls around a cache held to a budget at byte offsets past 2^32 (caches, workspaces,
scratch, weights, positions), and side by side on two streams. The definitions see compact
copies of what is used."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import budget_ops as bo
from oracle import kvarn_oracle as o
from tests.parity import assert_decode_close
from tests.test_budget_gpu import _axes_check, _evict, _make, _tiles, _weigh, env  # noqa: F401 (env: the fixture)
from tests.verify_common import record_pool, to_dev

pytestmark = pytest.mark.gpu

HKV = 8
REC = o.RECORD_BYTES
NUM_BLOCKS = 40000                            # 40000 x 8 x 14336 B = 4.59 GB
MARK31, MARK32 = (1 << 31) // (HKV * REC), (1 << 32) // (HKV * REC)
PLACES = [0, MARK31, MARK31 + 1, MARK32, MARK32 + 1, NUM_BLOCKS - 1]
FAR = 8300                                    # sequences: 8300 x 8 x 64 KB = 4.35 GB of workspace
WIDTH = 1100                                  # 8300 x 8 x 1100 tiles x 64 B = 4.67 GB of (m, l)


def test_weigh_past_4gb(env):
    kv, torch = env
    pool = record_pool("k4v2", len(PLACES), HKV, 0)
    cache = torch.zeros(NUM_BLOCKS, HKV, REC, dtype=torch.uint8, device="cuda")
    cache[torch.tensor(PLACES, device="cuda")] = to_dev(torch, pool)
    ws = torch.zeros(FAR, HKV, 2, 128, 128, dtype=torch.float16, device="cuda")
    used = {0: 300, 5: 0, FAR - 2: 128 * 6 + 77, FAR - 1: 5}
    small = sorted(used)
    lens = np.zeros(FAR, np.int32)
    lens[small] = [used[s] for s in small]
    small_ws = synth.workspace_tokens(len(small), HKV, seed=71)
    ws[torch.tensor(small, device="cuda")] = to_dev(torch, small_ws)
    bt, small_bt = np.full((FAR, WIDTH), -1, np.int32), np.full((len(small), WIDTH), -1, np.int32)
    for i, s in enumerate(small):
        n = used[s] // 128
        small_bt[i, :n] = np.roll(np.arange(6), i)[:n]
        bt[s, :n] = np.asarray(PLACES)[small_bt[i, :n]]
    q = np.zeros((FAR, 16, 128), np.float16)
    q[small] = synth.queries(len(small), 16, 72)
    weights = torch.full((FAR, HKV, WIDTH), 0.25, device="cuda")
    meta = kv.make_meta(HKV, 16, NUM_BLOCKS, max_blocks_per_seq=WIDTH)
    need = kv.decode_weights_scratch_bytes(meta, FAR)
    assert need > 1 << 32
    out = torch.empty(FAR, 16, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    kv.kvarn_decode_attention_weights(to_dev(torch, q), cache, ws, to_dev(torch, bt), to_dev(torch, lens), weights, out,
                                      scratch, meta, decay=0.5)
    assert kv.kvarn_device_flags() == 0
    before = np.full((len(small), HKV, WIDTH), 0.25, np.float32)
    want, _, w_want = bo.decode_weights(q[small], pool, small_ws, small_bt, lens[small], before, 0.5)
    at = torch.tensor(small, device="cuda")
    assert_decode_close(out[at].double().cpu().numpy(), want)
    got = weights[at].double().cpu().numpy()
    assert np.allclose(got, w_want, rtol=1e-3, atol=1e-9)
    weights[at] = 0.25
    assert bool((weights == 0.25).all()) and bool((out[1:5] == 0).all())


def test_evict_past_4gb(env):
    kv, torch = env
    rng = np.random.default_rng(73)
    pool = rng.integers(0, 256, (len(PLACES), HKV, REC), dtype=np.uint8)
    cache = torch.zeros(NUM_BLOCKS, HKV, REC, dtype=torch.uint8, device="cuda")
    at = torch.tensor(PLACES, device="cuda")
    cache[at] = to_dev(torch, pool)
    w = rng.random((2, HKV, 7)).astype(np.float32)
    small_bt = np.array([[5, 0, 3, 2, 4, 1, -1], [-1] * 7], np.int32)
    bt = np.where(small_bt < 0, -1, np.asarray(PLACES)[small_bt]).astype(np.int32)
    lens, budgets = np.array([6 * 128 + 9, 100], np.int32), np.array([3, 0], np.int32)
    d = [to_dev(torch, x) for x in (w, lens, bt, budgets)]
    wo, lo, kept = torch.empty_like(d[0]), torch.empty_like(d[1]), torch.empty(w.shape, dtype=torch.int32, device="cuda")
    kv.kvarn_evict_tiles(d[0], wo, d[1], lo, d[2], d[3], kept, cache, kv.make_meta(HKV, HKV, NUM_BLOCKS, 7), keep_first=1,
                         keep_last=1)
    assert kv.kvarn_device_flags() == 0
    want = bo.evict_tiles(w, lens, small_bt, budgets, pool, 1, 1)
    for a, b in zip((kept, lo, wo, cache[at]), want):
        assert np.array_equal(a.cpu().numpy(), b)
    cache[at] = 0
    assert not bool(cache.any())


def test_evict_with_weights_past_2_31_entries(env):
    kv, torch = env
    n, width = 33000, 8200
    assert n * HKV * width > 1 << 31
    rng = np.random.default_rng(74)
    pool = rng.integers(0, 256, (16, HKV, 10240), dtype=np.uint8)
    seqs = [0, 17000, n - 1]
    lens, budgets = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    bt = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(n, HKV, width, device="cuda")
    small_w = np.zeros((3, HKV, width), np.float32)
    small_w[:, :, :5] = rng.random((3, HKV, 5))
    small_bt = np.full((3, width), -1, np.int32)
    for i, s in enumerate(seqs):
        small_bt[i, :5] = np.arange(5) + 5 * i
        lens[s], budgets[s] = 5 * 128 + i, 2 + i
    bt[seqs], w[seqs] = to_dev(torch, small_bt), to_dev(torch, small_w)
    cache, lo, kept = to_dev(torch, pool), torch.empty_like(lens), torch.empty(n, HKV, width, dtype=torch.int32, device="cuda")
    kv.kvarn_evict_tiles(w, w, lens, lo, bt, budgets, kept, cache, kv.make_meta(HKV, HKV, 16, width, preset="k2v2"))
    assert kv.kvarn_device_flags() == 0
    want = bo.evict_tiles(small_w, [5 * 128 + i for i in range(3)], small_bt, [2, 3, 4], pool, 1, 1)
    for a, b in zip((kept[seqs], lo[seqs], w[seqs], cache), want):
        assert np.array_equal(a.cpu().numpy(), b)
    kept[seqs] = -1
    assert bool((kept == -1).all())


def test_axes_positions_past_4gb(env):
    kv, torch = env
    held = torch.zeros(2, 1 << 30, dtype=torch.int32, device="cuda")
    held[0, :5], held[1, :5] = 7, torch.arange(5, device="cuda") * 1000
    q, k = (torch.randn(5, h, 128, device="cuda").half() for h in (4, 2))
    inv = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    a, b = ([torch.empty_like(x) for x in (q, k)] for _ in range(2))
    axes, meta = [0] * 32 + [1] * 32, kv.make_meta(2, 4, 1, 1)
    kv.kvarn_qk_norm_rope_axes(q, k, None, held[:, :5], axes, *a, None, meta, inv_freq=inv)
    # (16-byte aligned rows of a small copy)
    near = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    near[:, :5] = held[:, :5]
    kv.kvarn_qk_norm_rope_axes(q, k, None, near[:, :5], axes, *b, None, meta, inv_freq=inv)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_streams(env):
    """A weighing decode and an eviction on each of two streams at once, as when alone."""
    kv, torch = env
    jobs = []
    for i in range(2):
        p = _make([4000 + 700 * i, 129, 900], 16, 2, seed=80 + i)
        want = _weigh(env, p, 0.5)
        meta = kv.make_meta(2, 16, p["cache"].shape[0], p["bt"].shape[1])
        d = {x: to_dev(torch, p[x]) for x in ("q", "cache", "ws", "bt", "lens", "w")}
        d["out"] = torch.empty(3, 16, 128, dtype=torch.float16, device="cuda")
        d["scratch"] = torch.empty(kv.decode_weights_scratch_bytes(meta, 3), dtype=torch.uint8, device="cuda")
        w, lens, bt, cache = _tiles([300, 200 + i, 64], 2, seed=82 + i)
        budgets = np.array([100, 199, 30], np.int32)
        ew = bo.evict_tiles(w, lens, bt, budgets, cache, 1, 2)
        e = [to_dev(torch, x) for x in (w, lens, bt, budgets, cache)]
        e += [torch.empty_like(e[0]), torch.empty_like(e[1]), torch.empty(w.shape, dtype=torch.int32, device="cuda")]
        jobs.append((meta, d, want, e, ew, kv.make_meta(2, 2, cache.shape[0], bt.shape[1], preset="k2v2"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for meta, d, _, e, _, m2, stream in jobs:
        for _ in range(2):
            kv.kvarn_decode_attention_weights(d["q"], d["cache"], d["ws"], d["bt"], d["lens"], d["w"], d["out"], d["scratch"],
                                              meta, decay=0.5, stream=stream)
        kv.kvarn_evict_tiles(e[0], e[5], e[1], e[6], e[2], e[3], e[7], e[4], m2, keep_first=1, keep_last=2, stream=stream)
    torch.cuda.synchronize()
    assert kv.kvarn_device_flags() == 0
    for meta, d, want, e, ew, _, _ in jobs:
        assert np.array_equal(d["out"].double().cpu().numpy(), want[0])
        for a, b in zip((e[7], e[6], e[5], e[4]), ew):
            assert np.array_equal(a.cpu().numpy(), b)


def test_all_at_once(env):
    """The most sequences of a call, and one of many more parts than tiles."""
    kv, torch = env
    n = 65535
    p = _make([200, 0, 300], 1, 1, seed=90)
    meta = kv.make_meta(1, 1, p["cache"].shape[0], p["bt"].shape[1])
    rep = n // 3
    d = {x: to_dev(torch, np.tile(p[x], (rep,) + (1,) * (p[x].ndim - 1))) for x in ("q", "bt", "lens", "w", "ws")}
    cache = to_dev(torch, p["cache"])
    out, lse = torch.empty(n, 1, 128, dtype=torch.float16, device="cuda"), torch.empty(n, 1, device="cuda")
    scratch = torch.empty(kv.decode_weights_scratch_bytes(meta, n), dtype=torch.uint8, device="cuda")
    kv.kvarn_decode_attention_weights(d["q"], cache, d["ws"], d["bt"], d["lens"], d["w"], out, scratch, meta, lse=lse)
    assert kv.kvarn_device_flags() == 0
    want, lse_want, w_want = bo.decode_weights(p["q"], p["cache"], p["ws"], p["bt"], p["lens"], p["w"])
    got = out.double().cpu().numpy().reshape(rep, 3, 1, 128)
    assert_decode_close(got, np.broadcast_to(want, got.shape))
    assert np.allclose(d["w"].double().cpu().numpy().reshape(rep, 3, 1, -1), w_want, rtol=1e-3)
    # equal sequences may be cut at different tiles: equal to the roundings of the join
    assert np.allclose(lse.double().cpu().numpy().reshape(rep, 3), lse_want[:, 0], atol=1e-4)
    w, lens, bt, c2 = _tiles([3] * 9, 1, seed=91)
    _evict(env, w, lens, bt, [1] * 9, c2, 0, 0)
