"""Host-side tests of the weight and eviction calls (no GPU): refusals, and launches in dry-run mode."""

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B

FAKE = 1 << 20


def _cache(dtype="bf16", hq=32, hkv=8, **kw):
    sc = None if dtype == "bf16" else FAKE
    return B.Cache(dtype, hq, hkv, **{**dict(k_pool=FAKE, v_pool=2 * FAKE, k_scale=sc, v_scale=sc, num_pages=4096), **kw})


class Plane:
    """A tensor's shape and address without the tensor."""

    def __init__(self, *shape, ptr=4 * FAKE):
        self.shape, self._p = shape, ptr

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self._p


def _mass(rows=((0, 999),), segs=None, cache=None, q=FAKE, lse=FAKE, cap=1024, decay=1.0, scale=0.088, ptr=4 * FAKE, nseg=None):
    segs = segs or [B.Seg(1000, page_table=3 * FAKE)]
    B.tfpa_key_mass(cache or _cache(), segs, q, lse, [r[0] for r in rows], [r[1] for r in rows], scale,
                    Plane(nseg or len(segs), 8, cap, ptr=ptr), decay=decay, stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.TFPA_EINVAL), (dict(q=FAKE + 4), B.TFPA_EINVAL), (dict(lse=None), B.TFPA_EINVAL), (dict(lse=FAKE + 2), B.TFPA_EINVAL),
    (dict(ptr=None), B.TFPA_EINVAL), (dict(ptr=FAKE + 1), B.TFPA_EINVAL), (dict(cap=999), B.TFPA_ECAPACITY), (dict(cap=0), B.TFPA_EINVAL),
    (dict(decay=-0.5), B.TFPA_EINVAL), (dict(decay=float("nan")), B.TFPA_EINVAL), (dict(decay=float("inf")), B.TFPA_EINVAL),
    (dict(scale=0.0), B.TFPA_EINVAL), (dict(scale=float("inf")), B.TFPA_EINVAL), (dict(rows=((1, 0),)), B.TFPA_ERANGE),
    (dict(rows=((0, 1000),)), B.TFPA_ERANGE), (dict(rows=((0, -1),)), B.TFPA_ERANGE), (dict(cache=_cache("fp4", k_scale=None)), B.TFPA_EINVAL)])
def test_mass_refusals(kw, code):
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        _mass(**kw)
    assert e.value.code == code and rec == []


def test_mass_shape_is_checked():
    with pytest.raises(ValueError):
        _mass(nseg=2)
    with pytest.raises(ValueError):
        B.tfpa_key_mass(_cache(), [B.Seg(1000, page_table=FAKE)], FAKE, FAKE, [0], [5], 0.1, torch.zeros(1, 1024, 8).transpose(1, 2))


def test_mass_launches():
    segs = [B.Seg(1000, page_table=3 * FAKE), B.Seg(300, page_table=3 * FAKE), B.Seg(128, k_slab=FAKE, v_slab=FAKE, slab_cap=256)]
    with B.record_launches() as rec:
        _mass(rows=[(0, 998), (0, 999), (2, 127), (1, 5), (0, 3)], segs=segs)
        _mass(rows=[], segs=segs)
    # a block per 128 keys and kv head; stream 0's two runs in one segment
    assert [(r["kind"], r["rows"], r["runs"], r["items"]) for r in rec] == [("key_mass", 5, 4, 8 * (8 + 3 + 1))]
    with B.record_launches() as rec:
        _mass(rows=[(0, p) for p in range(0, 400, 2)], segs=segs)      # 200 runs, 64 a launch
    assert [(r["rows"], r["runs"]) for r in rec] == [(64, 64)] * 3 + [(8, 8)]


def _evict(keep=(500,), segs=None, cap=1024, key_pos=None, next_pos=None, sink=0, recent=0, cache=None, mass=4 * FAKE, moves=5 * FAKE):
    segs = segs or [B.Seg(1000, page_table=3 * FAKE)]
    n = len(segs)
    kp = None if key_pos is None else Plane(n, 8, cap, ptr=key_pos)
    B.tfpa_evict_kv(cache or _cache(), segs, keep, Plane(n, 8, cap, ptr=mass), Plane(n, 8, cap + 4, ptr=moves), key_pos=kp,
                    next_pos=next_pos, sink=sink, recent=recent, stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(keep=[0]), B.TFPA_ERANGE), (dict(keep=[1001]), B.TFPA_ERANGE), (dict(cap=996), B.TFPA_ECAPACITY), (dict(cap=1001), B.TFPA_EINVAL),
    (dict(sink=-1), B.TFPA_EINVAL), (dict(recent=-1), B.TFPA_EINVAL), (dict(sink=300, recent=201), B.TFPA_EINVAL),
    (dict(sink=2**31 - 1, recent=2**31 - 1), B.TFPA_EINVAL), (dict(mass=None), B.TFPA_EINVAL), (dict(moves=None), B.TFPA_EINVAL),
    (dict(moves=FAKE + 8), B.TFPA_EINVAL), (dict(key_pos=FAKE + 2), B.TFPA_EINVAL), (dict(next_pos=[-1]), B.TFPA_ERANGE),
    (dict(cache=_cache("fp8", v_scale=None)), B.TFPA_EINVAL)])
def test_evict_refusals(kw, code):
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        _evict(**kw)
    assert e.value.code == code and rec == []


def test_evict_table_lengths_are_checked():
    for kw in (dict(keep=[1, 2]), dict(next_pos=[1, 2])):
        with pytest.raises(ValueError):
            _evict(**kw)


def test_evict_launches():
    with B.record_launches() as rec:
        _evict(sink=250, recent=250)
        _evict(keep=[1000], sink=2**31 - 1)                  # nothing to move, so nothing is checked against keep
    assert [(r["kind"], r["rows"], r["items"]) for r in rec] == [("evict", 1, 8), ("evict_move", 1, 8), ("evict", 1, 8)]
    segs = [B.Seg(300, page_table=3 * FAKE)] * 100
    with B.record_launches() as rec:
        _evict(keep=[100] * 100, segs=segs)
    assert [(r["kind"], r["row0"], r["rows"]) for r in rec] == [("evict", 0, 64), ("evict_move", 0, 64), ("evict", 64, 36), ("evict_move", 64, 36)]


def test_mass_of_more_tiles_than_a_launch_numbers():
    """A segment whose tiles pass 32 bits is refused; the launches before it are what they were."""
    L, hkv = 2 ** 31 - 257, 256
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        B.tfpa_key_mass(_cache(hq=hkv, hkv=hkv), [B.Seg(L, page_table=3 * FAKE)], FAKE, FAKE, [0], [5], 0.088,
                        Plane(1, hkv, L), stream=0)
    assert e.value.code == B.TFPA_ECAPACITY and rec == []
