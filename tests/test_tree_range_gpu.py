"""Attention of drafted tokens at the ends of its operands' ranges on the GPU, against its
float64 definition within the decode tolerance (tests/parity.py)."""
import numpy as np
import pytest

import kvarn_synth as synth
from oracle import kvarn_oracle as o
from oracle import verify_ops as vo
from tests.parity import assert_decode_close
from tests.test_tree_gpu import check, env, make, run  # noqa: F401 (env: the fixture)

pytestmark = pytest.mark.gpu


def quantized(k, v, preset):
    """Tiles [n, tokens, 128] of one kv-head as a cache of n blocks."""
    return o.quantize_tiles(np.asarray(k, np.float16)[:, None], np.asarray(v, np.float16)[:, None], preset=preset)[0]


@pytest.mark.parametrize("preset", ["k4v2", "k4v4", "k2v2", "k4v2l"])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size,noise,q_size,q_noise", [
    (5.0, 0.0, 12.0, 0.1), (1.9, 0.0, 1.9, 0.0), (24.0, 0.01, 30.0, 0.0), (250.0, 0.1, 12.0, 0.1), (6000.0, 1.0, 1.5, 0.0),
    (15.9, 0.0, 15.9, 0.0),
])
def test_keys_constant_in_one_channel(env, preset, sign, size, noise, q_size, q_noise):
    """Keys that are (nearly) the same number in one channel and nothing elsewhere, under queries
    along that channel: flat after the rotation, so that the zero points of all 128 channels add up with one
    sign, and far above the tile's steps."""
    rng = np.random.default_rng(140)
    p = make([300], [9], 8, 1, preset, seed=140)
    _, v = synth.prefill_kv(2 * 128, 1, seed=141)
    k = noise * rng.standard_normal((2, 128, 128))
    k[..., 5] += sign * size
    p["cache"], p["bt"] = quantized(k, v.reshape(2, 128, 128), preset), np.array([[0, 1, -1]], np.int32)
    q = q_noise * rng.standard_normal((9, 8, 128))
    q[..., 5] += q_size
    p["q"] = q.astype(np.float16)
    check(env, p)
