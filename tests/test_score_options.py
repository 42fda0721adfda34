"""Score options of the attention of drafted tokens that are refused, without a GPU."""
import pytest

from tests.test_verify_ops import _tree, kv  # noqa: F401 (kv: the fixture)


@pytest.mark.parametrize("size", [1e-45, 1e-40, 1.17e-38])
def test_subnormal_scales_and_caps_are_refused(kv, size):
    """A host in a mode that takes subnormal numbers for 0 would read them as the default scale, or no cap."""
    m = kv.make_meta(8, 64, 16, max_blocks_per_seq=4)
    for score in (kv.KvarnScore(size, 0, 0, 0, None), kv.KvarnScore(0, size, 0, 0, None)):
        assert _tree(kv, m, score) == 1
        assert "subnormal" in kv._lib.kvarn_last_error().decode()
    ok = kv.KvarnScore(1.2e-38, 1.2e-38, 0, 0, None)
    assert _tree(kv, m, ok, n=0) == 0
