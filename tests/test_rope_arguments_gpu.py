"""Arguments of the norm and rotation calls that the binding takes to the library, which refuses them."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def call():
    import torch
    import kv_cache_quantization_x128_gb300 as kv

    def one(axes, **more):
        q, k = (torch.ones(3, 1, 128, device="cuda").half() for _ in range(2))
        out = [torch.full((3, 1, 128), 7.0, device="cuda").half() for _ in range(2)]
        pos = torch.arange(3, dtype=torch.int32, device="cuda")
        inv, meta = torch.ones(64, device="cuda"), kv.make_meta(1, 1, 1, 1)
        if axes:
            kv.kvarn_qk_norm_rope_axes(q, k, None, pos.expand(2, 3), [0, 1] * 32, *out, None, meta, inv_freq=inv, **more)
        else:
            kv.kvarn_qk_norm_rope(q, k, None, pos, *out, None, meta, inv_freq=inv, **more)
        return out
    return kv, torch, one


@pytest.mark.parametrize("axes", [False, True])
@pytest.mark.parametrize("eps", [0.0, 1.0, -1e-6, 2.0, 1e39, -1e39, 1e-50, float("inf"), float("-inf"), float("nan")])
def test_norm_eps_out_of_range(call, axes, eps):
    kv, torch, one = call
    with pytest.raises(kv.KvarnError, match="norm_eps") as e:
        one(axes, norm_eps=eps)
    assert e.value.status == kv.KVARN_EINVAL


@pytest.mark.parametrize("axes", [False, True])
def test_norm_eps_as_numbers_of_other_types(call, axes):
    import numpy as np
    kv, torch, one = call
    want = one(axes, norm_eps=0.5)
    for eps in (np.float32(0.5), np.float64(0.5), torch.tensor(0.5)):
        assert all(torch.equal(x, y) for x, y in zip(want, one(axes, norm_eps=eps)))


def test_chunks_of_longer_rows_of_positions(call):
    """Columns of a prompt's positions: from a multiple of four tokens on, with rows at any stride; a copy elsewhere."""
    kv, torch, _ = call
    rows = torch.randint(0, 3000, (3, 101), dtype=torch.int32, device="cuda")
    inv, meta = (1e4 ** (-torch.arange(64, device="cuda") / 64)).float(), kv.make_meta(1, 2, 1, 1)
    axes = [i % 3 for i in range(64)]
    for start in range(12):
        n = 40 + start
        q, k = (torch.randn(n, h, 128, device="cuda").half() for h in (2, 1))
        got, want = ([torch.full_like(x, 7.0) for x in (q, k)] for _ in range(2))
        chunk = rows[:, start:start + n]
        kv.kvarn_qk_norm_rope_axes(q, k, None, chunk.clone(memory_format=torch.contiguous_format), axes, *want, None, meta,
                                   inv_freq=inv)
        if start % 4:
            with pytest.raises(kv.KvarnError, match="positions is not 16-byte aligned") as e:
                kv.kvarn_qk_norm_rope_axes(q, k, None, chunk, axes, *got, None, meta, inv_freq=inv)
            assert e.value.status == kv.KVARN_EALIGN
            assert all(bool((x == 7).all()) for x in got)
        else:
            kv.kvarn_qk_norm_rope_axes(q, k, None, chunk, axes, *got, None, meta, inv_freq=inv)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
