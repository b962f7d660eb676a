"""Host-side tests of the 4-bit cache (no GPU): refusals and launches in dry-run mode."""

import numpy as np
import pytest

from paged_kv_cache_235_gb300 import binding as B

FAKE = 1 << 20


def _cache(hq=32, hkv=8, **kw):
    return B.Cache("fp4", hq, hkv, **{**dict(k_pool=FAKE, v_pool=2 * FAKE, k_scale=FAKE, v_scale=FAKE, num_pages=64), **kw})


def _seg(L=1000, **kw):
    return B.Seg(L, page_table=3 * FAKE, **kw)


CALLS = {
    "write": lambda c, s: B.tfpa_write_kv(c, s, FAKE, FAKE, [0], [5], stream=0),
    "read": lambda c, s: B.tfpa_read_kv(c, s, FAKE, FAKE, [0], [5], stream=0),
    "decode": lambda c, s: B.tfpa_decode(c, s, FAKE, [0], [5], 0.088, B.Scratch(FAKE, FAKE, 4), FAKE, stream=0),
    "save": lambda c, s: B.tfpa_save_kv(c, s[0], 0, 5, FAKE, stream=0),
    "keep": lambda c, s: B.tfpa_keep_kv(c, s, [0], [1], [2], stream=0),
}


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("cache,seg,code", [
    (dict(k_scale=None), {}, B.TFPA_EINVAL), (dict(v_scale=None), {}, B.TFPA_EINVAL),
    (dict(k_pool=FAKE + 8), {}, B.TFPA_EINVAL), (dict(v_pool=None), {}, B.TFPA_EINVAL),
    (dict(hq=30), {}, B.TFPA_EINVAL), (dict(num_pages=0), {}, B.TFPA_EINVAL),
    ({}, dict(page_table_host=np.array([0, 1, 64, 2])), B.TFPA_ERANGE)])
def test_bad_caches_are_refused(call, cache, seg, code):
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        CALLS[call](_cache(**cache), [_seg(**seg)])
    assert e.value.code == code and rec == []


@pytest.mark.parametrize("args,code", [((FAKE + 2, FAKE, [0], [5]), B.TFPA_EINVAL), ((FAKE, None, [0], [5]), B.TFPA_EINVAL),
                                       ((FAKE, FAKE, [0], [1000]), B.TFPA_ERANGE), ((FAKE, FAKE, [1], [0]), B.TFPA_ERANGE)])
def test_read_refusals(args, code):
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        B.tfpa_read_kv(_cache(), [_seg()], *args, stream=0)
    assert e.value.code == code and rec == []


def test_read_launches():
    with B.record_launches() as rec:
        B.tfpa_read_kv(_cache(), [_seg(), _seg()], FAKE, FAKE, [0, 0, 1], [5, 6, 7], stream=0)
        B.tfpa_read_kv(_cache(), [_seg()], FAKE, FAKE, [], [], stream=0)
    assert [(r["kind"], r["rows"], r["runs"], r["grid"]) for r in rec] == [("read_kv", 3, 2, 2)]
    # more runs than a launch holds
    with B.record_launches() as rec:
        B.tfpa_read_kv(_cache(), [_seg()], FAKE, FAKE, [0] * 100, list(range(0, 200, 2)), stream=0)
    assert [(r["row0"], r["rows"], r["runs"]) for r in rec] == [(0, 64, 64), (64, 36, 36)]


def test_slab_capacity_is_in_positions():
    ok = B.Seg(300, k_slab=FAKE, v_slab=FAKE, slab_cap=512)
    bad = B.Seg(300, k_slab=FAKE, v_slab=FAKE, slab_cap=384)
    with B.record_launches() as rec:
        CALLS["decode"](_cache(), [ok])
    assert [r["kind"] for r in rec] == ["partial", "merge"]
    with B.record_launches(), pytest.raises(B.TfpaError) as e:
        CALLS["decode"](_cache(), [bad])
    assert e.value.code == B.TFPA_EINVAL


def test_runs_of_each_length_take_their_launches():
    """One decode call: up to 8 query vectors per kv head, up to 16, and more go to three kernels."""
    rs = np.repeat([0, 1, 2], [2, 4, 5])
    rp = np.concatenate([np.arange(998, 1000), np.arange(996, 1000), np.arange(995, 1000)])
    with B.record_launches() as rec:
        B.tfpa_decode(_cache(8, 2), [_seg() for _ in range(3)], FAKE, rs, rp, 0.1, B.Scratch(FAKE, FAKE, 64), FAKE, stream=0)
    kinds = [(r["kind"], r["runs"]) for r in rec]
    assert kinds[:2] == [("partial", 1)] * 2 and kinds[2:] == [("verify", 1), ("merge", 3)]


@pytest.mark.parametrize("rows,ok", [(1, True), (4, True), (5, False), (16, False)])
def test_device_mode_takes_the_decode_path_only(rows, ok):
    with B.record_launches():
        plan = B.Plan()
        assert B.lib().tfpa_plan_set_device(plan._p, FAKE, 1 << 16) == B.TFPA_OK
        args = (_cache(8, 2), [_seg()], FAKE, [0] * rows, list(range(1000 - rows, 1000)), 0.1, B.Scratch(FAKE, FAKE, 64), FAKE)
        if ok:
            plan.decode(*args)
            assert len(plan) == 2
        else:
            with pytest.raises(B.TfpaError) as e:
                plan.decode(*args)
            assert e.value.code == B.TFPA_EINVAL and len(plan) == 0
