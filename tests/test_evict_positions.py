"""Host-side refusals of positions that cannot be (no GPU)."""

import pytest

from paged_kv_cache_235_gb300 import binding as B
from tests.test_evict_host import FAKE, _evict


@pytest.mark.parametrize("key_pos", [None, 6 * FAKE])
@pytest.mark.parametrize("next_pos", [0, 500, 999])
def test_a_next_position_among_the_keys_is_refused(key_pos, next_pos):
    """seq_len keys at positions of their own below next_pos: next_pos is at least seq_len."""
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        _evict(next_pos=[next_pos], key_pos=key_pos)
    assert e.value.code == B.TFPA_ERANGE and rec == []


@pytest.mark.parametrize("key_pos", [None, 6 * FAKE])
@pytest.mark.parametrize("next_pos", [1000, 2 ** 31 - 1])
def test_a_next_position_behind_the_keys_is_taken(key_pos, next_pos):
    with B.record_launches() as rec:
        _evict(next_pos=[next_pos], key_pos=key_pos, recent=100)
    assert [r["kind"] for r in rec] == ["evict", "evict_move"]
