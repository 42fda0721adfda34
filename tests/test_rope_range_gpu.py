"""Norm and rotation of projected rows on the GPU: frequencies that are no numbers, and rows
whose strides do not count."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    import torch
    import kv_cache_quantization_x128_gb300 as kv
    torch.cuda.set_device(0)
    kv.kvarn_device_flags()
    return kv, torch


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,bad", [(128, (0, 63)), (64, (5,)), (16, (7, 2))])
def test_frequencies_that_are_no_numbers(env, rotary, bad, interleaved):
    """An angle of an infinite or undefined frequency is undefined at every position (0 too): so are the pair's two
    channels, and no other."""
    kv, torch = env
    n, half = 5, rotary // 2
    q, k, v = (torch.randn(n, h, 128, device="cuda").half() for h in (6, 2, 2))
    pos = torch.tensor([0, 1, 77, 100000, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    good = (1e4 ** (-torch.arange(half, device="cuda") / half)).float()
    meta = kv.make_meta(2, 6, 1, 1)
    want = [torch.empty_like(x) for x in (q, k, v)]
    kv.kvarn_qk_norm_rope(q, k, v, pos, *want, meta, inv_freq=good, interleaved=interleaved)
    for value in (float("nan"), float("inf"), -float("inf")):
        inv, got = good.clone(), [torch.empty_like(x) for x in (q, k, v)]
        inv[list(bad)] = value
        kv.kvarn_qk_norm_rope(q, k, v, pos, *got, meta, inv_freq=inv, interleaved=interleaved)
        hit = torch.zeros(128, dtype=torch.bool)
        for i in bad:
            hit[[2 * i, 2 * i + 1] if interleaved else [i, i + half]] = True
        for g, w in zip(got[:2], want[:2]):
            assert bool(torch.isnan(g[..., hit]).all()), value
            assert torch.equal(g[..., ~hit], w[..., ~hit])
        assert torch.equal(got[2], v)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_one_row_of_any_stride(env, dtype):
    """The stride between rows of a single row is no stride: tensors may carry any number there."""
    kv, torch = env
    t = getattr(torch, dtype)
    q, k, v = (torch.randn(1, h, 128, device="cuda").to(t) for h in (6, 2, 2))
    meta = kv.make_meta(2, 6, 1, 1)
    outs = [[torch.empty(1, h, 128, dtype=torch.float16, device="cuda") for h in (6, 2, 2)] for _ in range(2)]
    kv.kvarn_qk_norm_rope(q, k, v, None, *outs[0], meta)
    odd = [x.as_strided(x.shape, (s, 128, 1)) for x, s in zip((q, k, v), (1, 7, 130))]
    kv.kvarn_qk_norm_rope(*odd, None, *outs[1], meta)
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    none = [x.as_strided((0,) + x.shape[1:], (1, 128, 1)) for x in (q, k, v)]
    kv.kvarn_qk_norm_rope(*none, None, *[x[:0] for x in outs[1]], meta)
