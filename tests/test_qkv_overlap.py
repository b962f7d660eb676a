"""tfpa_write_qkv refuses a q_out that shares memory with any of its inputs, as its contract says (no GPU)."""

import pytest

from paged_kv_cache_235_gb300 import binding as B
from tests.test_blocks_host import FAKE, qkv, refused, tab

ROWS = ((0, 5), (0, 6), (0, 7))
OUT = 50 * FAKE
END = OUT + len(ROWS) * 32 * 256                  # bytes of q_out: rows x 32 heads x 128 bf16

INPUTS = {                                        # the input at an address, and its bytes
    "q_weight": (lambda p: dict(q_weight=p), 512),
    "k_weight": (lambda p: dict(k_weight=p), 512),
    "rope_cos": (lambda p: dict(rope_cos=tab(100, 32, p), rope_sin=tab(100, 32)), 100 * 32 * 4),
    "rope_sin": (lambda p: dict(rope_cos=tab(100, 32), rope_sin=tab(100, 32, p)), 100 * 32 * 4),
    "rope_pos": (lambda p: dict(rope_cos=tab(100, 32), rope_sin=tab(100, 32, 13 * FAKE), rope_pos=p), 12),
}


@pytest.mark.parametrize("name", INPUTS)
def test_q_out_shares_no_memory_with(name):
    make, size = INPUTS[name]
    step = 16                                     # an input's alignment
    first = (size + step - 1) // step * step      # the last place before q_out, and the first behind it, are free
    for p in (OUT, OUT - first + step, END - step, OUT + 1024):
        refused(B.TFPA_EINVAL, lambda: qkv(rows=ROWS, out=OUT, **make(p)))
    with B.record_launches() as rec:
        for p in (OUT - first, END):
            qkv(rows=ROWS, out=OUT, **make(p))
        qkv(rows=ROWS, q=0, out=0, **make(OUT))   # K and V only: there is no q_out
        qkv(rows=(), out=OUT, **make(OUT))
    assert len(rec) == 3


def test_inputs_that_are_not_read_do_not_count():
    """Rotary positions without a table."""
    with B.record_launches() as rec:
        qkv(rows=ROWS, out=OUT, rope_pos=OUT)
    assert len(rec) == 1
