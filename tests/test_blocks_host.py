"""Host-side tests of the calls from the projection to attention over selected blocks (no GPU): refusals, and
launches in dry-run mode."""

import os
import re

import pytest

from paged_kv_cache_235_gb300 import binding as B
from tests.test_evict_host import FAKE, Plane, _cache

LONG = B.Seg(5000, page_table=3 * FAKE)
SLAB = B.Seg(700, k_slab=FAKE, v_slab=FAKE, slab_cap=768)


class Rows(Plane):
    """Rows of heads at a stride, without their memory."""

    def __init__(self, rows, heads, ptr=8 * FAKE, stride=None, dense=True, head=128, last=1):
        super().__init__(rows, heads, 128, ptr=ptr)
        self._s, self._dense = (stride or heads * 128, head, last), dense

    def stride(self, i=None):
        return self._s if i is None else self._s[i]

    def is_contiguous(self):
        return self._dense


def refused(code, fn):
    with B.record_launches() as rec, pytest.raises(B.TfpaError) as e:
        fn()
    assert e.value.code == code and rec == []


# ---------------------------------------------------------------- tables
def table(first=0, n=16, cos=FAKE, sin=2 * FAKE, **kw):
    spec = B.RopeSpec(**{**dict(base=1e4), **kw})
    half = spec.rot_dim // 2
    B.tfpa_rope_table(spec, first, Plane(n, half, ptr=cos), Plane(n, half, ptr=sin), stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(base=1.0), B.TFPA_EINVAL), (dict(base=float("nan")), B.TFPA_EINVAL), (dict(base=float("inf")), B.TFPA_EINVAL),
    (dict(rot_dim=0), B.TFPA_EINVAL), (dict(rot_dim=8), B.TFPA_EINVAL), (dict(rot_dim=144), B.TFPA_EINVAL), (dict(rot_dim=40), B.TFPA_EINVAL),
    (dict(scaling="other"), B.TFPA_EINVAL), (dict(attn_scale=0.0), B.TFPA_EINVAL), (dict(attn_scale=float("inf")), B.TFPA_EINVAL),
    (dict(attn_scale=1e39), B.TFPA_EINVAL), (dict(attn_scale=1e-60), B.TFPA_EINVAL),
    (dict(scaling="linear", factor=0.5), B.TFPA_EINVAL), (dict(scaling="base", factor=float("nan")), B.TFPA_EINVAL),
    (dict(scaling="base", factor=1e300, base=1e300), B.TFPA_EINVAL),
    (dict(scaling="bands", factor=2.0, low=1.0, high=4.0), B.TFPA_EINVAL), (dict(scaling="ramp", factor=2.0, orig_len=100, low=4.0, high=4.0), B.TFPA_EINVAL),
    (dict(scaling="ramp", factor=2.0, orig_len=100, low=0.0, high=4.0), B.TFPA_EINVAL),
    (dict(cos=None), B.TFPA_EINVAL), (dict(sin=FAKE + 4), B.TFPA_EINVAL), (dict(first=-1), B.TFPA_ERANGE), (dict(first=2**31 - 15), B.TFPA_ERANGE),
    (dict(first=2**62), B.TFPA_ERANGE), (dict(first=2**63 - 1), B.TFPA_ERANGE)])
def test_table_refusals(kw, code):
    refused(code, lambda: table(**kw))


def test_table_launches():
    with B.record_launches() as rec:
        table(first=2**31 - 16)
        table(n=0, cos=None, sin=None)
        table(rot_dim=48, scaling="ramp", factor=4.0, orig_len=4096, low=1.0, high=32.0)
        table(factor=0.0)                                          # not read without a scaling
    assert [(r["kind"], r["rows"]) for r in rec] == [("rope_table", 16)] * 3
    with pytest.raises(ValueError):
        B.tfpa_rope_table(B.RopeSpec(1e4, rot_dim=32), 0, Plane(4, 64), Plane(4, 64))


# ---------------------------------------------------------------- a projection's rows
def qkv(rows=((0, 999),), q=8 * FAKE, k=9 * FAKE, v=10 * FAKE, out=11 * FAKE, cache=None, segs=None, hq=32, hkv=8, strides=(None,) * 3, **kw):
    n = len(rows)
    t = [None if p == 0 else Rows(n, h, p, s) for p, h, s in ((q, hq, strides[0]), (k, hkv, strides[1]), (v, hkv, strides[2]))]
    B.tfpa_write_qkv(cache or _cache(hq=hq, hkv=hkv), segs or [LONG], *t, None if out == 0 else Rows(n, hq, out), [r[0] for r in rows],
                     [r[1] for r in rows], stream=0, **kw)


def tab(n=2000, half=64, ptr=12 * FAKE):
    return Plane(n, half, ptr=ptr)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), B.TFPA_EINVAL), (dict(out=0), B.TFPA_EINVAL), (dict(q=FAKE + 8), B.TFPA_EINVAL), (dict(k=None), B.TFPA_EINVAL),
    (dict(v=FAKE + 2), B.TFPA_EINVAL), (dict(out=FAKE + 8), B.TFPA_EINVAL), (dict(q_weight=FAKE + 4), B.TFPA_EINVAL),
    (dict(k_weight=FAKE, eps=0.0), B.TFPA_EINVAL), (dict(q_weight=FAKE, eps=float("nan")), B.TFPA_EINVAL),
    (dict(rope_cos=tab(), rope_sin=tab(ptr=FAKE + 4)), B.TFPA_EINVAL), (dict(rope_cos=tab(ptr=FAKE + 8), rope_sin=tab()), B.TFPA_EINVAL),
    (dict(rope_cos=tab(), rope_sin=tab(ptr=None)), B.TFPA_EINVAL), (dict(rope_cos=tab(half=0), rope_sin=tab(half=0)), B.TFPA_EINVAL),
    (dict(rope_cos=tab(half=65), rope_sin=tab(half=65)), B.TFPA_EINVAL), (dict(rope_cos=tab(half=12), rope_sin=tab(half=12)), B.TFPA_EINVAL),
    (dict(rope_cos=tab(n=0), rope_sin=tab(n=0)), B.TFPA_EINVAL), (dict(rope_cos=tab(), rope_sin=tab(), rope_pos=FAKE + 2), B.TFPA_EINVAL),
    (dict(rope_cos=tab(n=999), rope_sin=tab(n=999)), B.TFPA_ERANGE), (dict(rows=((0, 5000),)), B.TFPA_ERANGE), (dict(rows=((1, 0),)), B.TFPA_ERANGE),
    (dict(cache=_cache("fp8", k_scale=None)), B.TFPA_EINVAL)])
def test_qkv_refusals(kw, code):
    refused(code, lambda: qkv(**kw))


@pytest.mark.parametrize("out,ok", [(8 * FAKE, False), (8 * FAKE + 32 * 256, False), (8 * FAKE + 48 * 256 + 47 * 256, False), (9 * FAKE, True)])
def test_q_out_shares_no_memory_with_a_fused_projection(out, ok):
    fused = dict(q=8 * FAKE, k=8 * FAKE + 32 * 256, v=8 * FAKE + 40 * 256, strides=(48 * 128,) * 3, rows=((0, 5), (0, 6)), out=out)
    if ok:
        with B.record_launches() as rec:
            qkv(**fused)
        assert len(rec) == 1
    else:
        refused(B.TFPA_EINVAL, lambda: qkv(**fused))


def test_q_out_may_be_q_itself():
    with B.record_launches() as rec:
        qkv(out=8 * FAKE, rows=((0, 5), (0, 6)))
        qkv(q=0, out=0)                                            # K and V only
    assert [(r["kind"], r["rows"], r["items"]) for r in rec] == [("write_qkv", 2, 80), ("write_qkv", 1, 8)]
    refused(B.TFPA_EINVAL, lambda: qkv(out=8 * FAKE, rows=((0, 5), (0, 6)), strides=(33 * 128, None, None)))
    refused(B.TFPA_EINVAL, lambda: qkv(out=8 * FAKE + 256, rows=((0, 5), (0, 6))))


@pytest.mark.parametrize("stride", [32 * 128 - 8, 32 * 128 + 4, 2**31])
def test_qkv_strides(stride):
    refused(B.TFPA_EINVAL, lambda: qkv(rows=((0, 5), (0, 6)), strides=(stride, None, None)))


def test_qkv_shapes_are_checked():
    good = Rows(1, 8, FAKE)
    for t in (Rows(1, 7, FAKE), Rows(2, 8, FAKE), Rows(1, 8, FAKE, head=256), Rows(1, 8, FAKE, last=2)):
        with pytest.raises(ValueError):
            B.tfpa_write_qkv(_cache(), [LONG], None, t, good, None, [0], [5], stream=0)
    with pytest.raises(ValueError):
        B.tfpa_write_qkv(_cache(), [LONG], Rows(1, 32), good, good, Rows(1, 31), [0], [5], stream=0)
    with pytest.raises(ValueError):
        qkv(rope_cos=tab(), rope_sin=tab(half=32))


def test_qkv_launches_are_cut_at_64_runs():
    with B.record_launches() as rec:
        qkv(rows=[(0, p) for p in range(0, 260, 2)], strides=(48 * 128,) * 3, q=20 * FAKE, k=40 * FAKE, v=60 * FAKE)
        qkv(rows=[])
    assert [(r["row0"], r["rows"], r["runs"], r["q_offset"], r["out_offset"]) for r in rec] == [
        (64 * i, n, n, 64 * i * 48 * 128, 64 * i * 32 * 128) for i, n in enumerate((64, 64, 2))]


# ---------------------------------------------------------------- bounds, selection, attention over blocks
def bounds(rows=((0, 999),), b=None, segs=None, cache=None):
    B.tfpa_key_bounds(cache or _cache(), segs or [LONG], b or B.Bounds(64, FAKE), [r[0] for r in rows], [r[1] for r in rows], stream=0)


def select(rows=((0, 999),), b=None, segs=None, cache=None, q=FAKE, nsel=16, blocks=2 * FAKE, sink=1, recent=2):
    B.tfpa_select_blocks(cache or _cache(), segs or [LONG], b or B.Bounds(64, FAKE), q, [r[0] for r in rows], [r[1] for r in rows],
                         Plane(len(rows), 8, nsel, ptr=blocks), sink=sink, recent=recent, stream=0)


def attend(rows=((0, 999),), segs=None, cache=None, q=FAKE, nsel=16, blocks=2 * FAKE, block=64, scale=0.088, out=3 * FAKE, lse=None):
    B.tfpa_decode_blocks(cache or _cache(), segs or [LONG], q, [r[0] for r in rows], [r[1] for r in rows], Plane(len(rows), 8, nsel, ptr=blocks),
                         block, scale, out, lse, stream=0)


BAD_BOUNDS = [B.Bounds(64, None), B.Bounds(64, FAKE + 8), B.Bounds(32, FAKE), B.Bounds(0, FAKE), B.Bounds(512, FAKE), B.Bounds(-64, FAKE)]


@pytest.mark.parametrize("i", range(len(BAD_BOUNDS)))
def test_bad_bounds_are_refused(i):
    refused(B.TFPA_EINVAL, lambda: bounds(b=BAD_BOUNDS[i]))
    refused(B.TFPA_EINVAL, lambda: select(b=BAD_BOUNDS[i]))


def test_slab_segments_need_bounds_of_their_own():
    segs = [LONG, SLAB]
    for b in (B.Bounds(64, FAKE), B.Bounds(64, FAKE, [FAKE, None]), B.Bounds(64, FAKE, [None, FAKE + 2])):
        refused(B.TFPA_EINVAL, lambda: bounds(rows=((1, 5),), b=b, segs=segs))
        refused(B.TFPA_EINVAL, lambda: select(rows=((1, 5),), b=b, segs=segs))
    with B.record_launches() as rec:
        bounds(rows=((1, 5), (0, 5)), b=B.Bounds(64, FAKE, [None, FAKE]), segs=segs)
        bounds(rows=((0, 5),), b=B.Bounds(64, FAKE), segs=segs)       # the slab has no row in the call
        select(rows=((1, 5),), b=B.Bounds(64, None, [None, FAKE]), segs=segs)
    assert [(r["kind"], r["runs"], r["items"]) for r in rec] == [("key_bounds", 2, 16), ("key_bounds", 1, 8), ("select_blocks", 1, 8)]
    with pytest.raises(ValueError):
        bounds(rows=((0, 5),), b=B.Bounds(64, FAKE, [None]), segs=segs)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.TFPA_EINVAL), (dict(q=FAKE + 4), B.TFPA_EINVAL), (dict(blocks=None), B.TFPA_EINVAL), (dict(blocks=FAKE + 2), B.TFPA_EINVAL),
    (dict(nsel=0, sink=0, recent=0), B.TFPA_EINVAL), (dict(sink=-1), B.TFPA_EINVAL), (dict(recent=-1), B.TFPA_EINVAL),
    (dict(sink=10, recent=7), B.TFPA_EINVAL), (dict(sink=2**31 - 1, recent=2**31 - 1), B.TFPA_EINVAL), (dict(rows=((0, 5000),)), B.TFPA_ERANGE),
    (dict(rows=((0, 18432 * 64),), segs=[B.Seg(2**21, page_table=FAKE)]), B.TFPA_ECAPACITY)])
def test_select_refusals(kw, code):
    refused(code, lambda: select(**kw))


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), B.TFPA_EINVAL), (dict(q=FAKE + 4), B.TFPA_EINVAL), (dict(blocks=None), B.TFPA_EINVAL), (dict(blocks=FAKE + 2), B.TFPA_EINVAL),
    (dict(out=None), B.TFPA_EINVAL), (dict(out=FAKE + 8), B.TFPA_EINVAL), (dict(lse=FAKE + 2), B.TFPA_EINVAL), (dict(nsel=0), B.TFPA_EINVAL),
    (dict(block=32), B.TFPA_EINVAL), (dict(block=192), B.TFPA_EINVAL), (dict(scale=0.0), B.TFPA_EINVAL), (dict(scale=float("nan")), B.TFPA_EINVAL),
    (dict(rows=((0, 5000),)), B.TFPA_ERANGE), (dict(rows=((0, -1),)), B.TFPA_ERANGE), (dict(cache=_cache("fp4", v_scale=None)), B.TFPA_EINVAL)])
def test_attend_refusals(kw, code):
    refused(code, lambda: attend(**kw))


def test_block_lists_shapes_are_checked():
    for shape in ((1, 7, 4), (2, 8, 4), (1, 8)):
        with pytest.raises(ValueError):
            B.tfpa_decode_blocks(_cache(), [LONG], FAKE, [0], [5], Plane(*shape), 64, 0.1, FAKE, stream=0)


def test_calls_with_their_arguments_in_memory():
    """tfpa_call does what the call that it names does, and refuses names that there are not."""
    import ctypes
    import numpy as np
    L = B.lib()
    c, n = _cache(), 2
    segs = B.SegTable([LONG])
    rs, rp = np.zeros(n, np.int32), np.array([999, 1000], np.int32)
    b = B.Bounds(64, FAKE).c()
    spec = B.RopeSpec(1e4).c()
    q = B.tfpa_qkv(8 * FAKE, 9 * FAKE, 10 * FAKE, 32 * 128, 8 * 128, 8 * 128, eps=1e-6)
    at = (ctypes.byref(c.c()), segs.arr, 1)
    rows = (rs.ctypes.data, rp.ctypes.data, n)
    with B.record_launches() as direct:
        assert L.tfpa_rope_table(ctypes.byref(spec), 7, n, FAKE, 2 * FAKE, 0) == 0
        assert L.tfpa_write_qkv(*at, ctypes.string_at(ctypes.byref(q), ctypes.sizeof(q)), *rows, 11 * FAKE, 0) == 0
        assert L.tfpa_key_bounds(*at, ctypes.byref(b), *rows, 0) == 0
        assert L.tfpa_select_blocks(*at, ctypes.byref(b), FAKE, *rows, 4, 1, 2, 2 * FAKE, 0) == 0
        assert L.tfpa_decode_blocks(*at, FAKE, *rows, 64, 4, 2 * FAKE, 0.1, 3 * FAKE, None, 0) == 0
    with B.record_launches() as rec:
        for op in range(5):
            a = B.tfpa_call_args(op=op, nseg=1, cache=ctypes.addressof(c.c()), segs=ctypes.addressof(segs.arr), row_seg=rows[0], row_pos=rows[1],
                                 bounds=ctypes.addressof(b), q=FAKE, blocks=2 * FAKE, out=11 * FAKE if op == 1 else 3 * FAKE, rows=n, block=64, nsel=4,
                                 sink=1, recent=2, softmax_scale=0.1)
            if op == 0:
                a.u.rope.spec, a.u.rope.first, a.u.rope.cos, a.u.rope.sin = ctypes.addressof(spec), 7, FAKE, 2 * FAKE
            else:
                a.u.qkv = q
            assert L.tfpa_call(ctypes.string_at(ctypes.byref(a), ctypes.sizeof(a))) == 0
    assert rec == direct and [r["kind"] for r in rec] == ["rope_table", "write_qkv", "key_bounds", "select_blocks", "decode_blocks"]
    with B.record_launches() as rec:
        for op in (-1, 5, 2**31 - 1):
            a.op = op
            assert L.tfpa_call(ctypes.string_at(ctypes.byref(a), ctypes.sizeof(a))) == B.TFPA_EINVAL
        assert L.tfpa_call(None) == B.TFPA_EINVAL
        a.op, a.softmax_scale = 4, 1e300                     # infinite as a float
        assert L.tfpa_call(ctypes.string_at(ctypes.byref(a), ctypes.sizeof(a))) == B.TFPA_EINVAL
    assert rec == []


def test_row_tables_of_other_kinds():
    """Lists, other integers, read-only and strided tables, and tables of two lengths."""
    import numpy as np
    frozen = np.array([998, 999], np.int32)
    frozen.flags.writeable = False
    for rs, rp in (([0, 0], [998, 999]), (np.zeros(2, np.int64), np.array([998, 999])), (np.zeros(2, np.int32), frozen),
                   (np.zeros(4, np.int32)[::2], np.array([998, 5, 999, 5], np.int32)[::2])):
        with B.record_launches() as rec:
            B.tfpa_key_bounds(_cache(), [LONG], B.Bounds(64, FAKE), rs, rp, stream=0)
        assert [(r["kind"], r["rows"], r["runs"]) for r in rec] == [("key_bounds", 2, 1)]
    for f in (lambda: B.tfpa_key_bounds(_cache(), [LONG], B.Bounds(64, FAKE), [0, 0], [5], stream=0),
              lambda: attend(rows=((0, 5),)) or B.tfpa_decode_blocks(_cache(), [LONG], FAKE, [0], [5, 6], Plane(1, 8, 4), 64, 0.1, FAKE, stream=0)):
        with B.record_launches(), pytest.raises(ValueError):
            f()


def test_elements_of_another_size_are_refused():
    """A tensor of narrower elements would be read or written past its end."""
    torch = pytest.importorskip("torch")
    half = torch.zeros(4, 64, dtype=torch.float16)
    full = torch.zeros(4, 64)
    for f in (lambda: B.tfpa_rope_table(B.RopeSpec(1e4), 0, half, half, stream=0),
              lambda: B.tfpa_rope_table(B.RopeSpec(1e4), 0, full, half, stream=0),
              lambda: qkv(rope_cos=full, rope_sin=half),
              lambda: qkv(rope_cos=full, rope_sin=full, rope_pos=torch.zeros(1, dtype=torch.int16)),
              lambda: qkv(rope_cos=full, rope_sin=full, rope_pos=torch.zeros(2, dtype=torch.int32)),
              lambda: B.tfpa_select_blocks(_cache(), [LONG], B.Bounds(64, FAKE), FAKE, [0], [5], torch.zeros(1, 8, 16, dtype=torch.int16)),
              lambda: B.tfpa_decode_blocks(_cache(), [LONG], FAKE, [0], [5], torch.zeros(1, 8, 16, dtype=torch.int16), 64, 0.1, FAKE)):
        with B.record_launches() as rec, pytest.raises(ValueError):
            f()
        assert rec == []


def test_bounds_of_the_blocks_that_rows_fall_into():
    with B.record_launches() as rec:
        bounds(rows=[(0, 63)])
        bounds(rows=[(0, 63), (0, 64)])
        bounds(rows=[(0, p) for p in range(1000, 1300)], b=B.Bounds(128, FAKE))
        bounds(rows=[])
    assert [(r["rows"], r["items"]) for r in rec] == [(1, 8), (2, 16), (300, 8 * 4)]


def test_the_longest_row_that_selection_takes():
    with B.record_launches() as rec:
        select(rows=((0, 18432 * 64 - 1),), segs=[B.Seg(2**21, page_table=FAKE)])
        select(rows=((0, 18432 * 256 - 1),), segs=[B.Seg(2**23, page_table=FAKE)], cache=_cache(num_pages=2**15), b=B.Bounds(256, FAKE))
    assert len(rec) == 2


@pytest.mark.parametrize("name", ["qkv.cu", "blocks.cu"])
def test_no_thread_leaves_its_role_alone(name):
    """As tests/test_wait_forms.py has it for the other kernels."""
    from tests.test_wait_forms import CSRC, alone, statements, strip
    with open(os.path.join(CSRC, name)) as f:
        src = strip(f.read())
    bad = [(line, s) for line, s, h in statements(src) if re.search(r"\bgoto\b", s) and alone(s, h)]
    assert not bad, bad


WAITS = ["attend_blocks.cu", "blocks.cu"]


@pytest.mark.parametrize("name", WAITS)
def test_a_warp_waits_as_one(name):
    """No lane waits, or leaves a loop, on an answer of its own: every wait is a whole warp's."""
    from tests.test_wait_forms import CSRC, WAIT, statements, strip
    with open(os.path.join(CSRC, name)) as f:
        src = strip(f.read())
    assert not [(line, s) for line, s, _ in statements(src) if WAIT.search(s)]
    waits = [s for _, s, _ in statements(src) if "warp_wait" in s]
    assert len(waits) == (3 if name == "attend_blocks.cu" else 0), waits


def test_loads_in_flight_land_before_a_block_ends():
    from tests.test_wait_forms import CSRC, strip
    with open(os.path.join(CSRC, "attend_blocks.cu")) as f:
        src = " ".join(strip(f.read()).split())
    assert src.count("if (sh.lost) let_copies_land();") == 1


# ---------------------------------------------------------------- host memory
def child(name):
    """As in tests/test_host_memory.py: a process whose address space leaves no room for a call's row groups."""
    import resource
    import numpy as np
    n = 8_000_000
    rs, rp = np.zeros(n, np.int32), np.zeros(n, np.int32)
    rp[1::2] = 5                                                 # no two rows in one group
    c = B.Cache("bf16", 8, 2, FAKE, FAKE, num_pages=64)
    segs = [B.Seg(1000, page_table=FAKE)]
    rows = lambda h, p: Rows(n, h, p)  # noqa: E731
    q, k, v, out = rows(8, FAKE), rows(2, FAKE), rows(2, FAKE), rows(8, 1 << 50)
    blocks, bnd = Plane(n, 2, 4, ptr=FAKE), B.Bounds(64, FAKE)
    calls = {
        "qkv": lambda: B.tfpa_write_qkv(c, segs, q, k, v, out, rs, rp, stream=0),
        "bounds": lambda: B.tfpa_key_bounds(c, segs, bnd, rs, rp, stream=0),
        "select": lambda: B.tfpa_select_blocks(c, segs, bnd, FAKE, rs, rp, blocks, stream=0),
        "attend": lambda: B.tfpa_decode_blocks(c, segs, FAKE, rs, rp, blocks, 64, 0.1, FAKE, stream=0),
    }
    with open("/proc/self/status") as f:
        size = next(int(x.split()[1]) for x in f if x.startswith("VmSize")) * 1024
    with B.record_launches() as rec:
        resource.setrlimit(resource.RLIMIT_AS, (size + (16 << 20), resource.RLIM_INFINITY))
        try:
            calls[name]()
            print("done")
        except B.TfpaError as e:
            print("code", e.code, len(rec), B.strerror(e.code))
        resource.setrlimit(resource.RLIMIT_AS, (resource.RLIM_INFINITY, resource.RLIM_INFINITY))


@pytest.mark.parametrize("name", ["qkv", "bounds", "select", "attend"])
def test_host_memory_that_runs_out_is_an_error_code(name):
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"from tests.test_blocks_host import child; child({name!r})"], cwd=root, capture_output=True,
                       text=True, timeout=120, env=dict(os.environ, OPENBLAS_NUM_THREADS="1", OMP_NUM_THREADS="1"))
    assert r.returncode == 0, (r.returncode, r.stderr[-600:])
    assert r.stdout.split()[:3] == ["code", str(B.TFPA_ENOMEM), "0"], r.stdout


def test_parts_of_a_list_follow_from_its_length_and_ctas_from_the_batch():
    """A part for every 128 keys, up to eight; a CTA takes as few as let the launch have four CTAs a SM (152 SMs here)."""
    segs = [B.Seg(60000, page_table=3 * FAKE)]
    c = _cache(num_pages=4096)

    def grids(rows, nsel, block=64):
        with B.record_launches() as rec:
            B.tfpa_decode_blocks(c, segs, FAKE, [0] * rows, list(range(50000, 50000 + rows)), Plane(rows, 8, nsel, ptr=FAKE), block, 0.1, FAKE,
                                 stream=0)
        return [(r["items"], r["grid"]) for r in rec]
    assert grids(1, 1) == [(8, 8)] and grids(1, 2) == [(8, 8)] and grids(1, 3) == [(8, 16)] and grids(1, 1, 256) == [(8, 16)]
    assert grids(1, 64) == [(8, 64)] and grids(8, 64) == [(64, 512)]
    assert grids(16, 64) == [(128, 512)] and grids(32, 64) == [(256, 512)] and grids(100, 64) == [(800, 800)]
    assert grids(32, 9) == [(256, 512)]                          # five parts: four in one CTA, one in the other
