"""The calls around a cache held to a budget, without a GPU: their float64 definitions
against each other and against worked examples, and the calls' refusals."""
import ctypes

import numpy as np
import pytest

import kvarn_synth as synth
from oracle import budget_ops as bo
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.test_library import A, B, MIS, kv  # noqa: F401 (kv: the fixture)
from tests.verify_common import paged


# ------------------------------------------------------------------ definitions
def test_axes_of_text_are_one_axis():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((4, 2, 128)), 1 + 0.2 * rng.standard_normal(128)
    inv = (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    pos = np.array([0, 5, 77, 100000])
    for inter in (False, True):
        one = vo.qk_norm_rope(x, w, 1e-6, inv, pos, inter)
        many = bo.qk_norm_rope_axes(x, w, 1e-6, inv, np.stack([pos] * 3), [i % 3 for i in range(32)], inter)
        assert np.array_equal(one, many)


def test_axes_turn_their_own_pairs():
    x = np.zeros((1, 1, 128))
    x[..., :8] = 1
    inv = np.ones(8, np.float32)
    pos = np.array([[0], [1]])
    y = bo.qk_norm_rope_axes(x, None, 1e-6, inv, pos, [0] * 4 + [1] * 4, False)[0, 0]
    assert np.array_equal(y[:4], np.ones(4)) and np.allclose(y[4:8], np.cos(1)) and np.allclose(y[12:16], np.sin(1))


def test_weights_of_tiles_sum_to_the_heads():
    lens = np.array([300, 128, 5, 0], np.int32)
    cache, bt, ws = paged("k4v2", lens, 2, 3)
    q = synth.queries(4, 6, 4)
    out, lse, w = bo.decode_weights(q, cache, ws, bt, lens, np.zeros((4, 2, bt.shape[1])))
    assert np.allclose(w.sum(2)[:3], 3) and (w[3] == 0).all() and (lse[3] == -np.inf).all()
    want = o.decode(q[:3], cache, ws, bt[:3], lens[:3])
    assert np.allclose(out[:3], want, atol=1e-12)
    _, _, again = bo.decode_weights(q, cache, ws, bt, lens, w, 0.5)
    assert np.allclose(again.sum(2)[:3], 4.5)


def test_evict_worked_example():
    # slots       0  1  2  3  4  5  6  7 (the partial tile: 8)
    w = np.array([[[9, 1, 5, 2, 7, 2, 8, 3, 4, 0]]], np.float32)
    cache = np.arange(10, dtype=np.uint8)[:, None, None].repeat(4, 2)
    bt = np.array([[3, 1, 0, 9, 2, 5, 6, 7, 4, -1]], np.int32)
    kept, lens, out, moved = bo.evict_tiles(w, [8 * 128 + 5], bt, [5], cache, 1, 2)
    # first 1, last 2 stay; of slots 1..5 the weights 7 and 5 do: slot 2 in place, slot 4 into slot 1
    assert kept[0, 0].tolist() == [0, 4, 2, 6, 7, 1, 3, 5, -1, -1]
    assert lens.tolist() == [5 * 128 + 5] and out[0, 0].tolist() == [9, 7, 5, 8, 3, 4, 0, 0, 0, 0]
    assert moved[bt[0, :5], 0, 0].tolist() == [3, 2, 0, 6, 7]
    # equal weights: the lowest slot stays
    kept = bo.evict_tiles(np.ones((1, 1, 6), np.float32), [6 * 128], bt[:, :6], [3], cache, 0, 1)[0]
    assert kept[0, 0].tolist() == [0, 1, 5, 2, 3, 4]


def test_attention_over_what_stays():
    """A decode over the evicted cache is one over the kept tokens alone."""
    lens = np.array([5 * 128 + 9], np.int32)
    cache, _, ws = paged("k4v2", lens, 1, 5)
    bt = np.array([[0, 1, 2, 3, 4, -1]], np.int32)
    q = synth.queries(1, 4, 6)
    _, _, w = bo.decode_weights(q, cache, ws, bt, lens, np.zeros((1, 1, 6)))
    kept, new, _, after = bo.evict_tiles(w, lens, bt, [3], cache, 1, 1)
    out, _, _ = bo.decode_weights(q, after, ws, bt, new, np.zeros((1, 1, 6)))
    k, v = vo.cached_tokens(cache, ws, bt[0], 0, int(lens[0]), 0)
    mine = np.concatenate([np.arange(t * 128, t * 128 + 128) for t in kept[0, 0, :3]] + [np.arange(640, 649)])
    assert np.allclose(out[0], o.attend(q[0].astype(np.float64), k[mine], v[mine]), atol=1e-12)


# ------------------------------------------------------------------ refusals
def _axes(kv, n=3, stride=16, axis=None, reserved=0):
    a = kv.KvarnAxes(n, reserved, stride)
    for i, x in enumerate(axis or [i % 3 for i in range(64)]):
        a.axis[i] = x
    return ctypes.byref(a)


def _call_axes(kv, axes, rope=None, n=16, **ptr):
    p = dict(q=A, k=A, v=A, qw=A, kw=A, inv=A, pos=A, qo=A, ko=A, vo=A) | ptr
    r = rope or kv.KvarnRope(kv.KVARN_F16, 128, 0, 1e-6, 8192, 1024, 1024)
    m = kv.make_meta(8, 64, 1)
    return kv._lib.kvarn_qk_norm_rope_axes(p["q"], p["k"], p["v"], ctypes.byref(r), axes, p["qw"], p["kw"], p["inv"],
                                           p["pos"], n, p["qo"], p["ko"], p["vo"], ctypes.byref(m), None)


def test_axes_refusals(kv):
    assert ctypes.sizeof(kv.KvarnAxes) == 80 and kv.KvarnAxes.position_stride.offset == 8
    assert _call_axes(kv, None) == 1
    assert _call_axes(kv, _axes(kv, n=0)) == 1 and _call_axes(kv, _axes(kv, n=5)) == 1
    assert _call_axes(kv, _axes(kv, n=2)) == 1                           # axis 2 of two
    assert _call_axes(kv, _axes(kv, axis=[0] * 63 + [3])) == 1
    assert _call_axes(kv, _axes(kv, reserved=1)) == 1
    assert _call_axes(kv, _axes(kv, stride=15)) == 1 and _call_axes(kv, _axes(kv, stride=-16)) == 1
    assert _call_axes(kv, _axes(kv), inv=None) == 1 and _call_axes(kv, _axes(kv), pos=None) == 1
    for name in ("q", "k", "qo", "ko", "vo"):
        assert _call_axes(kv, _axes(kv), **{name: None}) == 1, name
    for name in ("q", "k", "v", "qw", "kw", "inv", "pos", "qo", "ko", "vo"):
        assert _call_axes(kv, _axes(kv), **{name: MIS}) == 3, name
    assert _call_axes(kv, _axes(kv), n=-1) == 1 and _call_axes(kv, _axes(kv), n=1 << 31) == 1
    assert _call_axes(kv, _axes(kv), kv.KvarnRope(kv.KVARN_F16, 96, 0, 1e-6, 8192, 1024, 1024)) == 2
    # nothing to do; pairs behind the rotated ones are not looked at
    assert _call_axes(kv, _axes(kv), n=0) == 0
    part = kv.KvarnRope(kv.KVARN_F16, 32, 0, 1e-6, 8192, 1024, 1024)
    assert _call_axes(kv, _axes(kv, axis=[0] * 16 + [9] * 48), part, n=0) == 0


def _weigh(kv, m, n=4, short=0, decay=1.0, **ptr):
    p = dict(q=A, cache=A, ws=A, bt=A, lens=A, w=A, out=A, lse=A, scratch=A) | ptr
    need = kv.decode_weights_scratch_bytes(m, n) if 0 <= n <= 65535 else 1 << 30
    return kv._lib.kvarn_decode_attention_weights(p["q"], p["cache"], p["ws"], p["bt"], p["lens"], n, decay, p["w"],
                                                  p["out"], p["lse"], p["scratch"], need - short, ctypes.byref(m), None)


def test_weights_refusals(kv):
    m = kv.make_meta(8, 64, 16, max_blocks_per_seq=4)
    assert kv.decode_weights_scratch_bytes(m, 4) >= kv.decode_scratch_bytes(m, 4) + 4 * 8 * 4 * 64
    assert kv.decode_weights_scratch_bytes(m, -1) == kv.decode_weights_scratch_bytes(m, 65536) == 0
    for name in ("q", "cache", "bt", "lens", "w", "out", "scratch"):
        assert _weigh(kv, m, **{name: None}) == 1, name
        assert _weigh(kv, m, **{name: MIS}) == 3, name
    for name in ("ws", "lse"):
        assert _weigh(kv, m, **{name: MIS}) == 3, name
    assert _weigh(kv, m, n=-1) == 1 and _weigh(kv, m, n=65536) == 1 and _weigh(kv, m, short=1) == 4
    for decay in (-0.1, 1.01, float("nan"), float("inf"), 1e-40):
        assert _weigh(kv, m, decay=decay) == 1, decay
    assert _weigh(kv, m, n=0) == 0
    wide = kv.make_meta(1, 16, 16, max_blocks_per_seq=4)
    assert _weigh(kv, wide) == 2


def test_weights_out_over_q(kv):
    m, size = kv.make_meta(8, 64, 16, max_blocks_per_seq=4), 4 * 64 * 128 * 2
    q = 1 << 32
    for out in (q, q + 16, q - 16, q + size - 16, q - size + 16):
        assert _weigh(kv, m, q=ctypes.c_void_p(q), out=ctypes.c_void_p(out)) == 1, out - q
        assert b"overlap" in kv._lib.kvarn_last_error(), out - q


def test_evict_refusals(kv):
    def call(m=kv.make_meta(8, 64, 16, max_blocks_per_seq=4), n=4, first=1, last=1, **ptr):
        p = dict(w=A, wo=A, lens=A, lo=B, bt=A, budgets=A, kept=A, cache=A) | ptr
        return kv._lib.kvarn_evict_tiles(p["w"], p["wo"], p["lens"], p["lo"], p["bt"], p["budgets"], n, first, last,
                                         p["kept"], p["cache"], ctypes.byref(m), None)
    for name in ("w", "wo", "lens", "lo", "bt", "budgets", "kept", "cache"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: MIS}) == 3, name
    assert call(lo=A) == 1                                               # seq_lens_out aliases seq_lens
    assert call(n=-1) == 1 and call(n=65536) == 1 and call(first=-1) == 1 and call(last=-1) == 1
    assert call(kv.make_meta(8, 64, 16, max_blocks_per_seq=0)) == 1
    assert call(kv.make_meta(200, 200, 16, max_blocks_per_seq=4), n=65535) == 1    # 2^23 pairs and more
    assert call(n=0) == 0


def test_python_checks(kv):
    torch = pytest.importorskip("torch")
    m = kv.make_meta(1, 1, 1, 1)
    h, i32 = torch.zeros(2, 1, 128, dtype=torch.float16), torch.zeros(3, 2, dtype=torch.int32)
    inv = torch.ones(64)
    for pos in (i32[0], i32[:, :1], i32):                                # no axes; too short; not on a GPU
        with pytest.raises(ValueError):
            kv.kvarn_qk_norm_rope_axes(h, h, h, pos, [0] * 64, h, h, h, m, inv_freq=inv)
    f = torch.zeros(2, 1, 1)
    with pytest.raises(ValueError):
        kv.kvarn_evict_tiles(f, f, i32[0], i32[1], i32, i32[0], i32, h, m)
    with pytest.raises(ValueError):
        kv.kvarn_decode_attention_weights(h, h, None, i32, i32[0], f, h, h, m)
