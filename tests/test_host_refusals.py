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


@pytest.mark.parametrize("L", [2 ** 31 - 1, 2 ** 31 - 255, 2 ** 31 - 256])
@pytest.mark.parametrize("call", ["decode", "write", "mass"])
def test_a_stream_longer_than_its_slab_is_refused_whatever_its_length(L, call):
    """Lengths whose number of positions, rounded up to whole pages, passes 32 bits."""
    segs, c = [B.Seg(L, k_slab=FAKE, v_slab=FAKE, slab_cap=256)], _cache()
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        if call == "decode":
            B.tfpa_decode(c, segs, FAKE, [0], [5], 0.088, B.Scratch(FAKE, FAKE, 8, 32), FAKE, None, stream=0)
        elif call == "write":
            B.tfpa_write_kv(c, segs, FAKE, FAKE, [0], [1000], stream=0)
        else:
            B.tfpa_key_mass(c, segs, FAKE, FAKE, [0], [5], 0.088, Plane(1, 8, 2 ** 31 - 1), stream=0)
    assert e.value.code == B.TFPA_EINVAL and rec == []


def test_splits_of_the_longest_stream():
    assert [B.tfpa_num_splits(n) for n in (2 ** 31 - 1, 2 ** 31 - 256)] == [32, 32]
