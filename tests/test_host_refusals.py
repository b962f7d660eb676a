"""Calls that have to be refused whole, on the host (no GPU): nothing of them is enqueued."""

import pytest

from paged_kv_cache_235_gb300 import binding as B
from tests.test_evict_host import FAKE, Plane, _cache


def test_mass_of_a_batch_with_one_segment_too_long_enqueues_nothing():
    """The segments before the one whose tiles pass 32 bits are not summed first."""
    L, hkv = 2 ** 31 - 257, 256
    segs = [B.Seg(1000, page_table=3 * FAKE), B.Seg(L, page_table=3 * FAKE)]
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        B.tfpa_key_mass(_cache(hq=hkv, hkv=hkv), segs, FAKE, FAKE, [0, 1], [5, 5], 0.088, Plane(2, hkv, L), stream=0)
    assert e.value.code == B.TFPA_ECAPACITY and rec == []
