"""The calls around a verify step, without a GPU: their float64 definitions against
plainer ones, and their refusals (host-side, before any CUDA call)."""
import ctypes
import os

import numpy as np
import pytest

import kvarn_synth as synth
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.verify_common import paged, random_tree

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = ctypes.c_void_p(0x10000)          # aligned fake device address (never dereferenced)
MIS = ctypes.c_void_p(0x10008)        # not 16-byte aligned
B = ctypes.c_void_p(0x20000)


@pytest.fixture(scope="module")
def kv():
    import __graft_entry__
    if not os.path.exists(os.path.join(ROOT, "kv_cache_quantization_x128_gb300", "libkvarn.so")):
        __graft_entry__.build()
    import kv_cache_quantization_x128_gb300 as kv
    return kv


# ------------------------------------------------------------------ definitions
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [16, 64, 128])
def test_rotation_keeps_norms_and_relative_scores(interleaved, rotary):
    g = np.random.default_rng(1)
    x, y = g.standard_normal((2, 1, 2, 128))
    inv = (1e4 ** (-np.arange(rotary // 2) / (rotary // 2))).astype(np.float32)

    def rot(v, p):
        return vo.qk_norm_rope(v, None, 1e-6, inv, [p], interleaved)

    assert np.allclose(np.linalg.norm(rot(x, 12345), axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    s = (rot(x, 100) * rot(y, 93)).sum(-1)
    assert np.allclose(s, (rot(x, 1000007) * rot(y, 1000000)).sum(-1), atol=1e-9)   # only the distance counts
    assert np.array_equal(rot(x, 0), x)
    assert np.array_equal(rot(x, 5)[..., rotary:], x[..., rotary:])


def test_norm_definition():
    x = np.random.default_rng(2).standard_normal((3, 2, 128)) * 7
    y = vo.qk_norm_rope(x, np.full(128, 2.0), 1e-6, None, None, False)
    assert np.allclose((y ** 2).mean(-1), 4.0, rtol=1e-6)


def test_chain_is_chunked_prefill():
    lens, cu = [130, 5], np.array([0, 3, 7])
    cache, bt, ws = paged("k4v2", lens, 2, 3)
    q = synth.queries(7, 4, 3)
    k, v = synth.prefill_kv(7, 2, seed=3)
    want = o.prefill_attention(q.astype(np.float64), k, v, cu, np.array(lens), bt, ws, cache)
    got = vo.tree_attention(q, k, v, None, cu, lens, bt, ws, cache)
    assert np.allclose(got, want, atol=1e-12)


def test_tree_rows_are_their_paths():
    """A tree row equals the chain over its ancestors alone."""
    rng = np.random.default_rng(4)
    lens, cu = [140], np.array([0, 9])
    cache, bt, ws = paged("k2v2", lens, 1, 4)
    q, (k, v) = synth.queries(9, 2, 4), synth.prefill_kv(9, 1, seed=4)
    words, depths = random_tree(9, rng)
    pos = np.array([140 + d for d in depths])
    kw = dict(softcap=5.0, window=60, slopes=np.array([0.1, 0.02]))
    got = vo.tree_attention(q, k, v, words, cu, lens, bt, ws, cache, positions=pos, **kw)
    for t in range(9):
        path = [j for j in range(9) if words[t] >> j & 1]
        one = vo.tree_attention(q[path], k[path], v[path], None, np.array([0, len(path)]), lens, bt, ws, cache,
                                positions=pos[path], **kw)
        assert np.allclose(one[-1], got[t], atol=1e-12)


def test_append_tokens_is_append_repeated():
    lens = [126, 3]
    cache, bt, ws = paged("k4v2", lens, 1, 5, width=2)
    bt[:] = [[0, 1], [2, 3]]
    k, v = synth.prefill_kv(6, 1, seed=5)
    got = vo.append_tokens(k, v, [0, 3, 6], lens, bt, ws, cache)
    w, c, n = ws, cache, np.array(lens)
    for i in range(3):
        w, c, n = o.append(k[[i, 3 + i]], v[[i, 3 + i]], n, bt, w, c)
    assert np.array_equal(got[0], w) and np.array_equal(got[1], c) and np.array_equal(got[2], n)


def test_read_is_dequantization():
    lens = [300]
    cache, bt, ws = paged("k4v4", lens, 2, 6)
    k, v = vo.read_tokens(cache, ws, bt, lens, [100], [0, 200])
    kh, vh = o.dequant_record(cache[bt[0, 0], 1])
    assert np.allclose(k[:28, 1], kh.T[100:]) and np.allclose(v[:28, 1], vh.T[100:])
    assert np.array_equal(k[156:, 0], ws[0, 0, 0, :44].astype(np.float64))
    bound = vo.read_magnitude(cache, ws, bt, lens, [100], [0, 200], "k4v4")
    assert (np.abs(k[:156]).max(-1) <= bound[0][:156]).all() and (np.abs(v[:156]).max(-1) <= bound[1][:156]).all()


# ------------------------------------------------------------------ refusals
def _rope(kv, **change):
    r = kv.KvarnRope(kv.KVARN_F16, 128, 0, 1e-6, 8192, 1024, 1024)
    for name, value in change.items():
        setattr(r, name, value)
    return ctypes.byref(r)


def test_rope_struct_layout(kv):
    assert ctypes.sizeof(kv.KvarnRope) == 40 and kv.KvarnRope.q_stride.offset == 16


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), 2), (dict(rotary_dim=0), 2), (dict(rotary_dim=8), 2), (dict(rotary_dim=96), 2),
    (dict(interleaved=2), 1), (dict(norm_eps=0.0), 1), (dict(norm_eps=float("nan")), 1), (dict(q_stride=4096), 1),
    (dict(k_stride=1020), 1), (dict(k_stride=1028), 3), (dict(v_stride=-8), 1),
])
def test_rope_refuses_options(kv, change, status):
    m = kv.make_meta(8, 64, 1)
    f = kv._lib.kvarn_qk_norm_rope
    assert f(A, A, A, _rope(kv, **change), A, A, A, A, 2, A, A, A, ctypes.byref(m), None) == status
    assert kv._lib.kvarn_last_error().decode()


def test_rope_refuses_pointers_and_sizes(kv):
    m = ctypes.byref(kv.make_meta(8, 64, 1))
    f, r = kv._lib.kvarn_qk_norm_rope, _rope(kv)
    assert f(A, A, A, r, A, A, A, A, -1, A, A, A, m, None) == 1
    assert f(A, A, A, r, A, A, A, A, 1 << 31, A, A, A, m, None) == 1
    assert f(A, A, A, None, A, A, A, A, 1, A, A, A, m, None) == 1
    assert f(A, A, A, r, A, A, A, A, 1, A, A, A, None, None) == 1
    assert f(None, A, A, r, A, A, A, A, 1, A, A, A, m, None) == 1
    assert f(A, A, A, r, A, A, A, None, 1, A, A, A, m, None) == 1       # a rotation needs positions
    assert f(A, A, A, r, A, A, A, A, 1, A, A, None, m, None) == 1       # v without v_out
    assert f(A, A, A, r, MIS, A, A, A, 1, A, A, A, m, None) == 3
    assert f(A, MIS, A, r, A, A, A, A, 1, A, A, A, m, None) == 3
    assert f(None, None, None, r, None, None, None, None, 0, None, None, None, m, None) == 0


def _tree(kv, m, score=None, n=4, tokens=8, max_tree=4, short=0, **ptr):
    p = dict(q=A, k=A, v=A, mask=A, pos=A, cu=A, lens=A, bt=A, cache=A, ws=A, out=A, scratch=A) | ptr
    need = kv.tree_scratch_bytes(m, max(n, 0), max_tree) if 1 <= max_tree <= 64 else 1 << 20
    return kv._lib.kvarn_tree_attention(p["q"], p["k"], p["v"], p["mask"], p["pos"], p["cu"], p["lens"], n, tokens,
                                        max_tree, p["bt"], p["cache"], p["ws"],
                                        None if score is None else ctypes.byref(score), p["out"], p["scratch"],
                                        need - short, ctypes.byref(m), None)


def test_tree_refusals(kv):
    m = kv.make_meta(8, 64, 16, max_blocks_per_seq=4)
    S = kv.KvarnScore
    assert ctypes.sizeof(S) == 24 and S.slopes.offset == 16
    assert kv.tree_scratch_bytes(m, 4, 8) > 0
    assert kv.tree_scratch_bytes(m, 4, 0) == kv.tree_scratch_bytes(m, 4, 65) == kv.tree_scratch_bytes(m, -1, 4) == 0
    assert _tree(kv, m, max_tree=0) == 2 and _tree(kv, m, max_tree=65) == 2
    assert _tree(kv, m, n=-1) == 1 and _tree(kv, m, n=65536) == 1
    assert _tree(kv, m, tokens=-1) == 1 and _tree(kv, m, tokens=1 << 26) == 1
    assert _tree(kv, m, short=1) == 4 and _tree(kv, m, scratch=None) == 1 and _tree(kv, m, scratch=MIS) == 3
    for name in ("q", "k", "v", "cu", "lens", "bt", "cache", "out"):
        assert _tree(kv, m, **{name: None}) == 1, name
        assert _tree(kv, m, **{name: MIS}) == 3, name
    for name in ("mask", "pos", "ws"):
        assert _tree(kv, m, **{name: MIS}) == 3, name
    assert _tree(kv, m, S(0, 0, 5, 0, None), pos=None) == 1              # a window needs positions
    assert _tree(kv, m, S(0, 0, 0, 0, 0x10000), pos=None) == 1           # so do slopes
    assert _tree(kv, m, S(0, 0, 0, 0, 0x10008)) == 3
    for bad in (S(-1.0, 0, 0, 0, None), S(float("nan"), 0, 0, 0, None), S(float("inf"), 0, 0, 0, None),
                S(0, -1.0, 0, 0, None), S(0, float("inf"), 0, 0, None), S(0, 0, -1, 0, None), S(0, 0, 0, 1, None)):
        assert _tree(kv, m, bad) == 1
    assert _tree(kv, m, n=0) == 0 and _tree(kv, m, tokens=0) == 0


def test_append_tokens_refusals(kv):
    m = kv.make_meta(8, 64, 16, max_blocks_per_seq=4)
    f, r = kv._lib.kvarn_append_tokens, ctypes.byref(m)
    # k, v, cu, n_tokens, accepted, n_accepted, max_accept, lens, lens_out, bt, n_seqs, ws, cache, meta, stream
    assert f(A, A, A, 4, A, A, 2, A, A, A, 2, A, A, r, None) == 1        # seq_lens_out aliases seq_lens
    assert f(A, A, A, 4, A, None, 2, A, B, A, 2, A, A, r, None) == 1
    assert f(A, A, A, 4, None, A, 2, A, B, A, 2, A, A, r, None) == 1
    assert f(A, A, A, 4, A, A, -1, A, B, A, 2, A, A, r, None) == 1
    assert f(A, A, A, -1, A, A, 2, A, B, A, 2, A, A, r, None) == 1
    assert f(A, A, A, 4, A, A, 2, A, B, A, -1, A, A, r, None) == 1
    assert f(A, A, A, 4, A, A, 2, A, B, A, 1 << 21, A, A, r, None) == 1  # n_seqs * num_kv_heads * 256 rows beyond 2^31
    assert f(A, MIS, A, 4, A, A, 2, A, B, A, 2, A, A, r, None) == 3
    assert f(A, A, None, 4, A, A, 2, A, B, A, 2, A, A, r, None) == 1
    assert f(A, A, A, 4, A, A, 2, A, B, A, 2, None, A, r, None) == 1
    assert f(A, A, A, 4, A, A, 2, A, B, A, 0, A, A, r, None) == 0
    m0 = kv.make_meta(8, 64, 16, max_blocks_per_seq=0)
    assert f(A, A, A, 4, A, A, 2, A, B, A, 2, A, A, ctypes.byref(m0), None) == 1


def test_read_tokens_refusals(kv):
    m = kv.make_meta(8, 64, 16, max_blocks_per_seq=4)
    f, r = kv._lib.kvarn_read_tokens, ctypes.byref(m)
    # cache, ws, bt, lens, first, cu, n_seqs, n_tokens, dtype, k, v, meta, stream
    assert f(A, A, A, A, A, A, 2, 4, 3, A, A, r, None) == 2
    assert f(A, A, A, A, A, A, -1, 4, 0, A, A, r, None) == 1
    assert f(A, A, A, A, A, A, 2, -4, 0, A, A, r, None) == 1
    assert f(A, A, A, A, A, A, 2, 1 << 31, 0, A, A, r, None) == 1
    for i in (0, 2, 3, 5, 9, 10):
        args = [A, A, A, A, A, A, 2, 4, 0, A, A, r, None]
        args[i] = None
        assert f(*args) == 1, i
        args[i] = MIS
        assert f(*args) == 3, i
    assert f(A, A, A, A, A, A, 0, 4, 0, A, A, r, None) == 0
    assert f(A, A, A, A, A, A, 2, 0, 0, A, A, r, None) == 0


def test_python_checks(kv):
    torch = pytest.importorskip("torch")
    m = kv.make_meta(1, 1, 1, 1)
    h = torch.zeros(2, 1, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        kv.kvarn_qk_norm_rope(h, h, h, None, h, h, h, m)                 # not on a GPU
    with pytest.raises(ValueError):
        kv._heads(torch.zeros(2, 128), "q", 2, 1, torch.float32)
    with pytest.raises(ValueError):
        kv._heads(torch.zeros(2, 1, 256)[..., ::2], "q", 2, 1, torch.float32)
    with pytest.raises(ValueError):
        kv._dtype_code(torch.zeros(1, dtype=torch.float64), "q")
    assert kv._heads(torch.zeros(5, 384).unflatten(1, (3, 128))[:, 1:2], "k", 5, 1, torch.float32) == 384


@pytest.mark.parametrize("shape", [(2, 0), (3, 4), (2,)])
def test_python_refuses_rows_of_accepted_that_are_none(shape):
    torch = pytest.importorskip("torch")
    import kv_cache_quantization_x128_gb300 as kv
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    k = torch.zeros(4, 2, 128, dtype=torch.float16)
    ws = torch.zeros(2, 2, 2, 128, 128, dtype=torch.float16)
    with pytest.raises(ValueError, match="accepted must be"):
        kv.kvarn_append_tokens(k, k, i32(3), i32(2), i32(2), i32(2, 1), ws, torch.zeros(1, dtype=torch.uint8),
                               kv.make_meta(2, 2, 2, 1), accepted=i32(*shape), n_accepted=i32(2))
