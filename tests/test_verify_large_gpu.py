"""The calls around a verify step at byte offsets past 2^32 (caches, workspaces, rows), and side
by side on two streams. Every address formed from a block, sequence or token number has to be
64-bit for the first to pass; the second shares nothing but inputs. The oracle sees compact
copies of what is used."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.parity import assert_decode_close, compare_records
from tests.verify_common import HALF_STEP, TINY, paged, random_tree, record_pool, to_dev, words_to_dev

pytestmark = pytest.mark.gpu

HKV = 8
REC = o.RECORD_BYTES
NUM_BLOCKS = 40000                            # 40000 x 8 x 14336 B = 4.59 GB
MARK31, MARK32 = (1 << 31) // (HKV * REC), (1 << 32) // (HKV * REC)
PLACES = [0, MARK31, MARK31 + 1, MARK32, MARK32 + 1, NUM_BLOCKS - 1]
FAR = 8300                                    # sequences: 8300 x 8 x 64 KB = 4.35 GB of workspace


@pytest.fixture(scope="module")
def env():
    import torch
    import kv_cache_quantization_x128_gb300 as kv
    torch.cuda.set_device(0)
    kv.kvarn_device_flags()
    return kv, torch


@pytest.fixture(scope="module")
def big(env):
    """A cache past 2^32 bytes with six blocks in use, and a workspace past 2^32 bytes."""
    _, torch = env
    pool = record_pool("k4v2", len(PLACES), HKV, 0)
    cache = torch.zeros(NUM_BLOCKS, HKV, REC, dtype=torch.uint8, device="cuda")
    cache[torch.tensor(PLACES, device="cuda")] = to_dev(torch, pool)
    ws = torch.zeros(FAR, HKV, 2, 128, 128, dtype=torch.float16, device="cuda")
    assert (FAR - 2) * ws[0].numel() * 2 > 1 << 32
    return pool, cache, ws


def test_tree_and_read_past_4gb(env, big):
    kv, torch = env
    pool, cache, ws = big
    used = {0: 300, 5: 0, FAR - 2: 128 * 6 + 77, FAR - 1: 5}            # sequence -> cached tokens
    lens, counts = np.zeros(FAR, np.int32), np.zeros(FAR, np.int32)
    for s, n in used.items():
        lens[s], counts[s] = n, 1 + s % 4
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    small = sorted(used)
    small_ws = synth.workspace_tokens(len(small), HKV, seed=91)
    ws[torch.tensor(small, device="cuda")] = to_dev(torch, small_ws)
    bt, small_bt = np.full((FAR, 6), -1, np.int32), np.full((len(small), 6), -1, np.int32)
    for i, s in enumerate(small):
        n = used[s] // 128
        small_bt[i, :n] = np.roll(np.arange(6), i)[:n]
        bt[s, :n] = np.asarray(PLACES)[small_bt[i, :n]]
    n = int(cu[-1])
    q = synth.queries(n, 16, 92)
    k, v = synth.prefill_kv(n, HKV, seed=93)
    rng = np.random.default_rng(94)
    words = sum((random_tree(int(counts[s]), rng)[0] for s in small), [])
    meta = kv.make_meta(HKV, 16, NUM_BLOCKS, max_blocks_per_seq=6)
    out = torch.zeros(n, 16, 128, dtype=torch.float16, device="cuda")
    scratch = torch.empty(kv.tree_scratch_bytes(meta, FAR, 4), dtype=torch.uint8, device="cuda")
    d = {x: to_dev(torch, y) for x, y in dict(q=q, k=k, v=v, cu=cu, lens=lens, bt=bt).items()}
    kv.kvarn_tree_attention(d["q"], d["k"], d["v"], words_to_dev(torch, words), d["cu"], d["lens"], 4, d["bt"], cache, ws,
                            out, scratch, meta)
    assert kv.kvarn_device_flags() == 0
    small_cu = np.concatenate([[0], np.cumsum(counts[small])])
    want = vo.tree_attention(q, k, v, words, small_cu, lens[small], small_bt, small_ws, pool)
    assert_decode_close(out.double().cpu().numpy(), want)
    # the same tokens read back
    rcu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    for t in ("float16", "float32"):
        ko, vo_ = (torch.empty(int(rcu[-1]), HKV, 128, dtype=getattr(torch, t), device="cuda") for _ in range(2))
        kv.kvarn_read_tokens(cache, ws, d["bt"], d["lens"], to_dev(torch, rcu), ko, vo_, meta)
        assert kv.kvarn_device_flags() == 0
        scu, zero = np.concatenate([[0], np.cumsum(lens[small])]), np.zeros(len(small), int)
        want = vo.read_tokens(pool, small_ws, small_bt, lens[small], zero, scu)
        mag = vo.read_magnitude(pool, small_ws, small_bt, lens[small], zero, scu, "k4v2")
        for got, ref, m in zip((ko, vo_), want, mag):      # (tolerance: tests/test_verify_gpu.py)
            tol = HALF_STEP[t] * np.abs(ref) + TINY[t] + 12 * 2.0 ** -24 * m[:, :, None]
            assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()


def test_append_past_4gb(env, big):
    kv, torch = env
    _, cache, ws = big
    lens, counts = np.zeros(FAR, np.int32), np.zeros(FAR, np.int32)
    lens[FAR - 1], counts[FAR - 1] = 126, 5
    lens[FAR - 2], counts[FAR - 2] = 127, 2
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    bt = np.full((FAR, 6), -1, np.int32)
    bt[FAR - 1, 0], bt[FAR - 2, 0] = NUM_BLOCKS - 2, MARK32 + 2
    tail = synth.workspace_tokens(2, HKV, seed=95)
    ws[FAR - 2:] = to_dev(torch, tail)
    k, v = synth.prefill_kv(7, HKV, seed=96)
    meta = kv.make_meta(HKV, HKV, NUM_BLOCKS, max_blocks_per_seq=6)
    out = torch.zeros(FAR, dtype=torch.int32, device="cuda")
    kv.kvarn_append_tokens(to_dev(torch, k), to_dev(torch, v), to_dev(torch, cu), to_dev(torch, lens), out,
                           to_dev(torch, bt), ws, cache, meta)
    assert kv.kvarn_device_flags() == 0
    small_bt = np.full((2, 6), -1, np.int32)
    small_bt[:, 0] = [0, 1]
    want_ws, _, want_lens, done = vo.append_tokens(k, v, cu[FAR - 2:], lens[FAR - 2:], small_bt, tail,
                                                   np.zeros((2, HKV, REC), np.uint8))
    assert np.array_equal(out.cpu().numpy()[FAR - 2:], want_lens)
    assert np.array_equal(ws[FAR - 2:].view(torch.int16).cpu().numpy().view(np.float16), want_ws)
    for _, blk, tile in done:
        _, kq, vq = o.quantize_tiles(tile[:, 0], tile[:, 1])
        compare_records(cache[[MARK32 + 2, NUM_BLOCKS - 2][blk]].cpu().numpy(), kq, vq)


def test_read_output_past_4gb(env):
    kv, torch = env
    tiles, hkv = 17000, HKV                                 # 2.18 M tokens: 4.46 GB a tensor
    n = tiles * 128 + 9
    cache = record_pool("k4v2", 6, hkv, 1)
    bt = np.random.default_rng(97).integers(0, 6, (1, tiles)).astype(np.int32)
    ws = synth.workspace_tokens(1, hkv, seed=98)
    meta = kv.make_meta(hkv, hkv, 6, max_blocks_per_seq=tiles)
    i32 = lambda a: to_dev(torch, np.asarray(a, np.int32))
    ko, vo_ = (torch.empty(n, hkv, 128, dtype=torch.float16, device="cuda") for _ in range(2))
    kv.kvarn_read_tokens(to_dev(torch, cache), to_dev(torch, ws), to_dev(torch, bt), i32([n]), i32([0, n]), ko, vo_, meta)
    assert kv.kvarn_device_flags() == 0
    m = 2 * 128 + 9                                         # the last two packed tiles and the workspace's tokens
    sbt = bt[:, -2:]
    want = vo.read_tokens(cache, ws, sbt, [m], [0], [0, m])
    mag = vo.read_magnitude(cache, ws, sbt, [m], [0], [0, m], "k4v2")
    for got, ref, mg in zip((ko, vo_), want, mag):
        tol = HALF_STEP["float16"] * np.abs(ref) + TINY["float16"] + 12 * 2.0 ** -24 * mg[:, :, None]
        assert (np.abs(got[-m:].double().cpu().numpy() - ref) <= tol).all()


def test_rope_rows_past_4gb(env):
    kv, torch = env
    n, hq, hkv = 270000, 64, 8                              # q: 4.42 GB in, 4.42 GB out
    g = torch.Generator(device="cuda").manual_seed(99)
    q = torch.randn(n, hq, 128, generator=g, device="cuda", dtype=torch.float16)
    k = torch.randn(n, hkv, 128, generator=g, device="cuda", dtype=torch.float16)
    w = torch.rand(128, generator=g, device="cuda", dtype=torch.float32).half() + 0.5
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    inv = (1e6 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    kv.kvarn_qk_norm_rope(q, k, None, pos, qo, ko, None, kv.make_meta(hkv, hq, 1, 1), q_weight=w, k_weight=w, inv_freq=inv)
    for x, out in ((q, qo), (k, ko)):
        rows = slice(n - 3, n)
        want = vo.qk_norm_rope(x[rows].double().cpu().numpy(), w.double().cpu().numpy(), 1e-6, inv.double().cpu().numpy(),
                               pos[rows].cpu().numpy(), False)
        raw = vo.qk_norm_rope(x[rows].double().cpu().numpy(), w.double().cpu().numpy(), 1e-6, None, None, False)
        got = out[rows].double().cpu().numpy()
        # (tolerance: tests/test_verify_gpu.py)
        tol = HALF_STEP["float16"] * np.abs(want) + TINY["float16"] + 2.0 ** -18 * np.abs(raw).max(-1, keepdims=True)
        assert (np.abs(got - want) <= tol).all()


def test_two_streams(env):
    """A tree call and a read of the same cache on each of two streams, over and over: scratch and
    outputs are each stream's own, results the same bits as alone."""
    kv, torch = env
    lens, counts = [1000, 130, 4000, 65], [8, 3, 1, 6]
    cache, bt, ws = paged("k4v2", lens, HKV, 100)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(cu[-1])
    k, v = synth.prefill_kv(n, HKV, seed=101)
    meta = kv.make_meta(HKV, 64, len(cache), max_blocks_per_seq=bt.shape[1])
    rcu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    d = [to_dev(torch, a) for a in (synth.queries(n, 64, 102), k, v, cu, np.asarray(lens, np.int32), bt, cache, ws, rcu)]

    def buffers():
        return dict(out=torch.zeros(n, 64, 128, dtype=torch.float16, device="cuda"),
                    k=torch.zeros(int(rcu[-1]), HKV, 128, dtype=torch.bfloat16, device="cuda"),
                    v=torch.zeros(int(rcu[-1]), HKV, 128, dtype=torch.bfloat16, device="cuda"),
                    scratch=torch.empty(kv.tree_scratch_bytes(meta, 4, 8), dtype=torch.uint8, device="cuda"))

    def step(b, stream=None):
        kv.kvarn_tree_attention(d[0], d[1], d[2], None, d[3], d[4], 8, d[5], d[6], d[7], b["out"], b["scratch"], meta,
                                stream=stream)
        kv.kvarn_read_tokens(d[6], d[7], d[5], d[4], d[8], b["k"], b["v"], meta, stream=stream)

    alone = buffers()
    step(alone)
    torch.cuda.synchronize()
    streams, each = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, b in zip(streams, each):
            step(b, s)
    torch.cuda.synchronize()
    assert kv.kvarn_device_flags() == 0
    for b in each:
        for x in ("out", "k", "v"):
            assert torch.equal(b[x], alone[x])
