"""kvarn_evict_tiles refuses outputs that lie over its inputs or over one another (no GPU: refused before any launch)."""
import ctypes

import pytest

from tests.test_library import kv  # noqa: F401 (the fixture)

SEQS, HKV, WIDTH = 4, 8, 12
ROWS, TABLE, ENTRIES = 4 * SEQS, 4 * SEQS * WIDTH, 4 * SEQS * WIDTH * HKV
SIZES = dict(weights=ENTRIES, weights_out=ENTRIES, seq_lens=ROWS, seq_lens_out=ROWS, block_tables=TABLE, budgets=ROWS,
             kept=ENTRIES)
OUTS = ("weights_out", "seq_lens_out", "kept")


def _call(kv, n=SEQS, **at):
    p = {name: at.get(name, 0x10000000 * (i + 1)) for i, name in enumerate((*SIZES, "cache"))}
    m = kv.make_meta(HKV, 64, 16, max_blocks_per_seq=WIDTH)
    ptr = {name: ctypes.c_void_p(x) for name, x in p.items()}
    return kv._lib.kvarn_evict_tiles(ptr["weights"], ptr["weights_out"], ptr["seq_lens"], ptr["seq_lens_out"],
                                     ptr["block_tables"], ptr["budgets"], n, 1, 1, ptr["kept"], ptr["cache"],
                                     ctypes.byref(m), None)


@pytest.mark.parametrize("out,other", [(out, other) for out in OUTS for other in SIZES if out != other])
def test_outputs_over_other_buffers(kv, out, other):  # noqa: F811
    base = 1 << 34
    # the same start, the last 16 bytes of the other one, and the output's own last 16 bytes
    for at in (base, base + SIZES[other] - 16, base - SIZES[out] + 16):
        if {out, other} == {"weights", "weights_out"} and at == base:
            continue                               # weights_out may be weights
        assert _call(kv, **{other: base, out: at}) == kv.KVARN_EINVAL, at - base
        assert b"must not overlap" in kv._lib.kvarn_last_error()


def test_weights_in_place_and_the_list_over_them(kv):  # noqa: F811
    base = 1 << 34
    assert _call(kv, weights=base, weights_out=base, kept=base) == kv.KVARN_EINVAL
    assert _call(kv, weights=base, weights_out=base, kept=base + 16) == kv.KVARN_EINVAL
    assert b"weights_out must not overlap kept" == kv._lib.kvarn_last_error()
    assert _call(kv, n=0, weights=base, weights_out=base, kept=base) == kv.KVARN_OK
