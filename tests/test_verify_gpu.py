"""Norm and rotation, the append of several tokens and the reading back of cached tokens
on the GPU, against their float64 definitions."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.parity import compare_records
from tests.verify_common import HALF_STEP, TINY, paged, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import kv_cache_quantization_x128_gb300 as kv
    torch.cuda.set_device(0)
    kv.kvarn_device_flags()
    return kv, torch


# ------------------------------------------------------------------ norm and rotation
def _rope_check(env, n, hq, hkv, dtype, norm=True, rotary=128, interleaved=False, fused=True, far=5000, in_place=False,
                with_v=True, positions=None, stream=None):
    kv, torch = env
    g = torch.Generator().manual_seed(n * 31 + hq)
    t = getattr(torch, dtype)
    x = (torch.randn(n, (hq + 2 * hkv) * 128 + 64, generator=g) * 3).to(t).cuda()
    q, k, v = (p.unflatten(1, (-1, 128)) for p in x[:, :-64].split([hq * 128, hkv * 128, hkv * 128], 1))
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    qw, kw = ((1 + 0.3 * torch.randn(128, generator=g)).to(t).cuda() if norm else None for _ in range(2))
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32) if positions is None else \
        torch.tensor(positions, dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(rotary // 2) / (rotary // 2))).float() if rotary else None
    want, plain = [], []
    for p, w in ((q, qw), (k, kw)):
        a = p.cpu().double().numpy()
        ww = None if w is None else w.cpu().double().numpy()
        want.append(vo.qk_norm_rope(a, ww, 1e-6, None if inv is None else inv.numpy(), pos.numpy(), interleaved))
        plain.append(vo.qk_norm_rope(a, ww, 1e-6, None, None, False))
    want.append(v.cpu().double().numpy())
    plain.append(want[2])
    outs = [q, k, v] if in_place else [torch.full((n, h, 128), 7.0, dtype=torch.float16, device="cuda")
                                       for h in (hq, hkv, hkv)]
    meta = kv.make_meta(hkv, hq, 1, 1)
    torch.cuda.synchronize()
    kv.kvarn_qk_norm_rope(q, k, v if with_v else None, pos.cuda() if rotary else None, outs[0], outs[1],
                          outs[2] if with_v else None, meta, q_weight=qw, k_weight=kw,
                          inv_freq=None if inv is None else inv.cuda(), interleaved=interleaved, stream=stream)
    torch.cuda.synchronize()
    if not with_v:
        assert bool((outs[2] == 7).all())
    for out, ref, raw in list(zip(outs, want, plain))[: 3 if with_v else 2]:
        # one rounding to fp16, and fp32 arithmetic before it: the mean square (127 sums of a
        # tree 12 deep), 1/sqrt, two products, sine and cosine (an angle to 2 pi 2^-25, 2 ulp),
        # two products and a sum: below 32 roundings of 2^-24 of each of a pair's magnitudes
        pair = np.abs(raw).max(-1, keepdims=True) if rotary else np.abs(raw)
        tol = 2.0 ** -11 * np.abs(ref) + TINY["float16"] + 2.0 ** -19 * 2 * pair
        err = np.abs(out.double().cpu().numpy() - ref)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 32, 64, 128])
def test_rope_types(env, dtype, interleaved, rotary):
    _rope_check(env, 7, 5, 1, dtype, rotary=rotary, interleaved=interleaved)


@pytest.mark.parametrize("n,hq,hkv", [(1, 64, 8), (1, 1, 1), (2, 8, 1), (37, 28, 4), (303, 40, 8), (1217, 6, 2),
                                      (2501, 16, 2)])
def test_rope_sizes(env, n, hq, hkv):
    _rope_check(env, n, hq, hkv, "float16")


def test_rope_without_parts(env):
    _rope_check(env, 9, 8, 2, "bfloat16", norm=False)
    _rope_check(env, 9, 8, 2, "float16", rotary=0)
    _rope_check(env, 9, 8, 2, "float32", norm=False, rotary=0, fused=False)
    _rope_check(env, 9, 8, 2, "float16", with_v=False)
    _rope_check(env, 1300, 3, 1, "float16", with_v=False, norm=False)


def test_rope_in_place(env):
    _rope_check(env, 40, 8, 2, "float16", fused=False, in_place=True)


def test_rope_far_positions(env):
    _rope_check(env, 6, 2, 1, "float16", positions=[0, 1, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1])


def test_rope_stream_and_graph(env):
    kv, torch = env
    side = torch.cuda.Stream()
    _rope_check(env, 33, 8, 2, "float16", stream=side)
    q, k, v = (torch.randn(5, h, 128, device="cuda").half() for h in (8, 2, 2))
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    inv = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float()
    a = [torch.empty_like(x) for x in (q, k, v)]
    b = [torch.empty_like(x) for x in (q, k, v)]
    meta = kv.make_meta(2, 8, 1, 1)
    kv.kvarn_qk_norm_rope(q, k, v, pos, *a, meta, inv_freq=inv)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kvarn_qk_norm_rope(q, k, v, pos, *b, meta, inv_freq=inv)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_rope_overflow_is_infinity(env):
    kv, torch = env
    x = torch.full((1, 1, 128), 1e6, dtype=torch.float32, device="cuda")
    out = torch.empty(1, 1, 128, dtype=torch.float16, device="cuda")
    kv.kvarn_qk_norm_rope(x, x, x, None, out, out.clone(), out.clone(), kv.make_meta(1, 1, 1, 1))
    assert bool(torch.isinf(out).all())


# ------------------------------------------------------------------ append
def _append(env, preset, lens, counts, hkv=2, seed=50, accepted=None, n_accepted=None, width=None, lens_out=True,
            expect=0, bt=None):
    kv, torch = env
    n = len(lens)
    width = width or max((x + 128) // 128 for x in lens) + 1
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k, v = synth.prefill_kv(max(int(cu[-1]), 1), hkv, seed=seed)
    ws = synth.workspace_tokens(n, hkv, seed=seed)
    if bt is None:
        bt = synth.block_tables(n, width, n * width, seed=seed)
    rec = o.LAYOUTS[preset].record_bytes
    cache = np.full((n * width, hkv, rec), 3, np.uint8)
    meta = kv.make_meta(hkv, hkv, n * width, max_blocks_per_seq=width, preset=preset)
    ws_d, cache_d = to_dev(torch, ws), to_dev(torch, cache)
    out = torch.full((n,), -7, dtype=torch.int32, device="cuda") if lens_out else None
    kv.kvarn_append_tokens(to_dev(torch, k), to_dev(torch, v), to_dev(torch, cu),
                           to_dev(torch, np.asarray(lens, np.int32)), out, to_dev(torch, bt), ws_d, cache_d, meta,
                           accepted=None if accepted is None else to_dev(torch, np.asarray(accepted, np.int32)),
                           n_accepted=None if n_accepted is None else to_dev(torch, np.asarray(n_accepted, np.int32)))
    assert kv.kvarn_device_flags() == expect
    got_ws = ws_d.view(torch.int16).cpu().numpy().view(np.float16)
    return (k, v, cu, ws, bt, cache), got_ws, cache_d.cpu().numpy(), None if out is None else out.cpu().numpy()


def _append_check(env, preset, lens, counts, accepted=None, n_accepted=None, **kw):
    (k, v, cu, ws, bt, cache), got_ws, got_cache, got_lens = _append(env, preset, lens, counts, accepted=accepted,
                                                                     n_accepted=n_accepted, **kw)
    want_ws, _, want_lens, done = vo.append_tokens(k, v, cu, lens, bt, ws, cache, accepted=accepted,
                                                   n_accepted=n_accepted)
    assert np.array_equal(got_ws, want_ws)
    if got_lens is not None:
        assert np.array_equal(got_lens, want_lens)
    for _, blk, tile in done:
        _, kq, vq = o.quantize_tiles(tile[:, 0], tile[:, 1], preset=preset)
        compare_records(got_cache[blk], kq, vq)
    keep = np.ones(len(got_cache), bool)
    keep[[blk for _, blk, _ in done]] = False
    assert (got_cache[keep] == 3).all()
    return len(done)


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
def test_append_whole_chunks(env, preset):
    # none; inside a tile; ending it; over its end; a whole tile from slot 0 and from slot 1; over the end by 127
    lens = [5, 5, 120, 125, 0, 129, 255, 127, 256]
    counts = [0, 3, 8, 9, 128, 128, 128, 1, 127]
    assert _append_check(env, preset, lens, counts) == 6


def test_append_accepted(env):
    lens = [100, 126, 127, 383, 0]
    acc = [[0, 2, 5, 7], [1, 3, 4, 6], [7, 0, 0, 3], [2, 9, 9, 9], [9, 9, 9, 9]]
    n_acc = [4, 3, 4, 1, 0]          # entries behind n_acc are not read; order and repeats are kept
    assert _append_check(env, "k4v2", lens, [8] * 5, accepted=np.array(acc), n_accepted=np.array(n_acc)) == 3


def test_append_without_lengths_out(env):
    assert _append_check(env, "k4v2", [126], [4], lens_out=False) == 1


def test_append_many_sequences(env):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 700, 200).astype(int).tolist()
    counts = rng.integers(0, 9, 200).tolist()
    _append_check(env, "k4v2", lens, counts, hkv=1)


def test_append_more_items_than_ranked(env):
    """More (sequence, kv-head) items than are handed out by rank (32768): 5 sequences complete a tile."""
    kv, torch = env
    n, hkv = 4100, 8
    at = [0, 700, 701, 2050, 4099]
    lens, counts = np.full(n, 3, np.int32), np.full(n, 1, int)
    lens[at], counts[at] = 126, [2, 3, 3, 4, 5]
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    k, v = synth.prefill_kv(int(cu[-1]), hkv, seed=51)
    g = torch.Generator(device="cuda").manual_seed(51)
    ws = torch.randn(n, hkv, 2, 128, 128, generator=g, device="cuda").half()
    before = ws.clone()
    bt = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    meta = kv.make_meta(hkv, hkv, n, max_blocks_per_seq=1, preset="k2v2")
    cache = torch.full((n, hkv, kv.meta_record_bytes(meta)), 3, dtype=torch.uint8, device="cuda")
    out = torch.zeros(n, dtype=torch.int32, device="cuda")
    kd, vd = to_dev(torch, k), to_dev(torch, v)
    kv.kvarn_append_tokens(kd, vd, to_dev(torch, cu), to_dev(torch, lens), out, bt, ws, cache, meta)
    assert kv.kvarn_device_flags() == 0
    assert np.array_equal(out.cpu().numpy(), lens + counts)
    one = np.setdiff1d(np.arange(n), at)
    i = torch.from_numpy(one).cuda()
    c = torch.from_numpy(cu[one].astype(np.int64)).cuda()
    before[i, :, 0, 3], before[i, :, 1, 3] = kd[c], vd[c]
    for s in at:
        tile = before[s].clone()
        tile[:, 0, 126:], tile[:, 1, 126:] = kd[cu[s]:cu[s] + 2].transpose(0, 1), vd[cu[s]:cu[s] + 2].transpose(0, 1)
        _, kq, vq = o.quantize_tiles(*(tile[:, x].view(torch.int16).cpu().numpy().view(np.float16) for x in (0, 1)),
                                     preset="k2v2")
        compare_records(cache[s].cpu().numpy(), kq, vq)
        m = counts[s] - 2
        tile[:, 0, :m], tile[:, 1, :m] = (x[cu[s] + 2:cu[s + 1]].transpose(0, 1) for x in (kd, vd))
        before[s] = tile
    assert torch.equal(ws, before)
    assert bool((cache[i] == 3).all())


def test_append_bad_numbers(env):
    kv, _ = env
    # a count over max_accept, a negative one, a negative length: nothing appended
    (k, v, cu, ws, *_), got, cache, lens = _append(
        env, "k4v2", [126, 10, -5, 7], [4] * 4, accepted=np.zeros((4, 3), int), n_accepted=np.array([4, -1, 1, 2]), width=2,
        expect=kv.FLAG_BAD_LENGTH)
    assert np.array_equal(got[:3], ws[:3]) and (cache == 3).all()
    assert lens.tolist() == [126, 10, -7, 9]
    assert np.array_equal(got[3, :, 0, 7], k[cu[3]]) and np.array_equal(got[3, :, 0, 8], k[cu[3]])
    # chunks of more than 128 rows are refused as a whole
    *_, lens = _append(env, "k4v2", [0, 0], [129, 2], width=2, expect=kv.FLAG_BAD_LENGTH)
    assert lens.tolist() == [0, 2]


def test_append_bad_index_keeps_its_slot(env):
    kv, _ = env
    (k, v, cu, ws, *_), got, _, lens = _append(env, "k4v2", [10, 20], [4, 4], accepted=np.array([[0, 4, 1], [-1, 2, 3]]),
                                                n_accepted=np.array([3, 3]), expect=kv.FLAG_BAD_INDEX)
    assert lens.tolist() == [13, 23]
    assert np.array_equal(got[0, :, 0, 10], k[0]) and np.array_equal(got[0, :, 1, 12], v[1])
    assert np.array_equal(got[0, :, 0, 11], ws[0, :, 0, 11]) and np.array_equal(got[1, :, 0, 20], ws[1, :, 0, 20])


def test_append_bad_block(env):
    kv, _ = env
    bt = np.array([[77, 1], [2, 3]], np.int32)
    (k, v, cu, ws, *_), got, cache, lens = _append(env, "k4v2", [126, 126], [4, 4], width=2, bt=bt,
                                                   expect=kv.FLAG_BAD_BLOCK)
    assert lens.tolist() == [130, 130]
    assert (cache[[0, 1, 3]] == 3).all() and not (cache[2] == 3).all()
    assert np.array_equal(got[0, :, 0, 1], k[3])                 # the tokens behind the lost tile are there
    _append(env, "k4v2", [254], [4], width=1, expect=kv.FLAG_BAD_LENGTH)   # block index beyond the table's row


# ------------------------------------------------------------------ reading back
def _read_check(env, preset, dtype, lens, first, counts, hkv=2, seed=60):
    kv, torch = env
    cache, bt, ws = paged(preset, lens, hkv, seed)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(cu[-1])
    t = getattr(torch, dtype)
    k, v = (torch.full((n + 3, hkv, 128), 9.0, dtype=t, device="cuda") for _ in range(2))
    meta = kv.make_meta(hkv, hkv, len(cache), max_blocks_per_seq=bt.shape[1], preset=preset)
    kv.kvarn_read_tokens(to_dev(torch, cache), to_dev(torch, ws), to_dev(torch, bt),
                         to_dev(torch, np.asarray(lens, np.int32)), to_dev(torch, cu), k, v, meta,
                         first=None if first is None else to_dev(torch, np.asarray(first, np.int32)))
    assert kv.kvarn_device_flags() == 0
    first = [0] * len(lens) if first is None else first
    want = vo.read_tokens(cache, ws, bt, lens, first, cu)
    mag = vo.read_magnitude(cache, ws, bt, lens, first, cu, preset)
    for out, ref, m in zip((k, v), want, mag):
        assert bool((out[n:] == 9).all())
        # the output's rounding, and fp32 arithmetic before it (12 roundings: r s, r z, the
        # code's fma twice, 7 butterfly stages, the final products) of the row's magnitude
        tol = HALF_STEP[dtype] * np.abs(ref) + TINY[dtype] + 12 * 2.0 ** -24 * m[:, :, None]
        err = np.abs(out[:n].double().cpu().numpy() - ref)
        assert (err <= tol).all(), (err / tol).max()


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_read_types(env, preset, dtype):
    _read_check(env, preset, dtype, [300, 128, 77], [100, 0, 3], [200, 128, 74])


@pytest.mark.parametrize("lens,first,counts", [
    ([1], None, [1]), ([128], [127], [1]), ([129], [127], [2]), ([129], [128], [1]), ([700], [250], [9]),
    ([0, 500, 0, 131], [0, 130, 0, 0], [0, 300, 0, 131]), ([384] * 5, None, [0, 1, 128, 129, 384]),
])
def test_read_ranges(env, lens, first, counts):
    _read_check(env, "k4v2", "float16", lens, first, counts, hkv=3)


def test_read_many_sequences(env):
    rng = np.random.default_rng(61)
    lens = rng.integers(1, 500, 75)
    counts = np.minimum(lens, rng.integers(0, 200, 75))
    first = [int(rng.integers(0, a - c + 1)) for a, c in zip(lens, counts)]
    _read_check(env, "k2v2", "float16", lens.tolist(), first, counts.tolist(), hkv=1)


def test_read_what_is_not_there(env):
    kv, torch = env
    lens = [300, 200, 300]
    cache, bt, ws = paged("k4v2", lens, 1, 62)
    bt[2, 1] = 99
    cu = np.array([0, 10, 20, 320], np.int32)
    k, v = (torch.full((320, 1, 128), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    meta = kv.make_meta(1, 1, len(cache), max_blocks_per_seq=bt.shape[1])
    args = [to_dev(torch, x) for x in (cache, ws, bt, np.asarray(lens, np.int32), cu)]
    first = to_dev(torch, np.array([295, -4, 0], np.int32))
    kv.kvarn_read_tokens(*args, k, v, meta, first=first)
    assert kv.kvarn_device_flags() == kv.FLAG_BAD_LENGTH | kv.FLAG_BAD_BLOCK
    for out in (k, v):
        old = (out == 9).all(-1)[:, 0].cpu().numpy()
        want = np.zeros(320, bool)
        want[5:10] = True                 # behind the length
        want[10:14] = True                # before token 0
        want[20 + 128:20 + 256] = True    # the bad block
        assert np.array_equal(old, want)
    # no workspace; fewer output rows than the last offset
    k.fill_(9.0)
    args[1] = None
    kv.kvarn_read_tokens(*args, k[:60], v[:60], meta, first=to_dev(torch, np.array([250, 0, 0], np.int32)))
    assert kv.kvarn_device_flags() == kv.FLAG_BAD_LENGTH
    old = (k == 9).all(-1)[:, 0].cpu().numpy()
    assert not old[:6].any() and old[6:10].all() and not old[10:60].any() and old[60:].all()


def test_read_is_what_quantize_wrote(env):
    """Tiles quantized by the library read back within the quantizer's own error, and bit for bit the same from a graph."""
    kv, torch = env
    k, v = synth.prefill_kv(256, 2, seed=63)
    kd, vd = to_dev(torch, k), to_dev(torch, v)
    meta = kv.make_meta(2, 2, 4, max_blocks_per_seq=2, preset="k4v4")
    cache = torch.zeros(4, 2, kv.meta_record_bytes(meta), dtype=torch.uint8, device="cuda")
    slots = torch.cat([torch.arange(384, 512), torch.arange(0, 128)]).cuda()
    kv.kvarn_quantize_tiles(kd, vd, slots, cache, meta)
    bt = torch.tensor([[3, 0]], dtype=torch.int32, device="cuda")
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([256], [0, 256]))
    a, b, c, d = (torch.empty_like(kd) for _ in range(4))
    kv.kvarn_read_tokens(cache, None, bt, lens, cu, a, b, meta)
    for got, ref in ((a, kd), (b, vd)):
        rel = ((got.float() - ref.float()).norm() / ref.float().norm()).item()
        assert rel < 0.12, rel            # 4-bit grid: a step of about 0.35 sigma, rounding error 0.1 sigma
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kvarn_read_tokens(cache, None, bt, lens, cu, c, d, meta)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d) and kv.kvarn_device_flags() == 0
