"""Host-side tests of what the Python calls from the projection to attention over selected blocks hand to the
library, and of what they refuse before they call it (no GPU)."""

import ctypes

import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests.test_blocks_host import FAKE, LONG, SLAB, bounds, select
from tests.test_evict_host import _cache


# ---------------------------------------------------------------- bounds of slabs
def handed(b, segs, monkeypatch):
    """The slab pointers that a call of bounds and a call of selection hand to the library."""
    got = []

    class Lib:
        @staticmethod
        def tfpa_call(args):
            a = B.tfpa_call_args.from_buffer_copy(args.ljust(ctypes.sizeof(B.tfpa_call_args), b"\0"))
            c = B.tfpa_bounds.from_address(a.bounds)
            got.append([x or 0 for x in (ctypes.c_void_p * a.nseg).from_address(c.slabs)])
            return 0

    with monkeypatch.context() as m:
        m.setattr(B, "lib", lambda: Lib)
        for f in (bounds, select):
            f(rows=((1, 5),), b=b, segs=segs)
    assert got[0] == got[1]
    return got[0]


def test_entries_changed_in_the_list_are_the_ones_used(monkeypatch):
    """A serving loop keeps the list, replaces its entries and lets it grow with the segments."""
    b = B.Bounds(64, FAKE, [None, FAKE])
    assert handed(b, [LONG, SLAB], monkeypatch) == [0, FAKE]
    b.slabs[1] = 5 * FAKE
    assert handed(b, [LONG, SLAB], monkeypatch) == [0, 5 * FAKE]
    b.slabs.append(6 * FAKE)
    assert handed(b, [LONG, SLAB, SLAB], monkeypatch) == [0, 5 * FAKE, 6 * FAKE]
    del b.slabs[0]
    assert handed(b, [SLAB, SLAB], monkeypatch) == [5 * FAKE, 6 * FAKE]
    b.slabs = [FAKE, None]
    assert handed(b, [SLAB, LONG], monkeypatch) == [FAKE, 0]


def test_what_a_call_was_handed_lives_until_it_is_over(monkeypatch):
    """Another thread changes the list while the library reads the entries (a call drops the interpreter's lock)."""
    b = B.Bounds(64, FAKE, [None, FAKE])
    seen = []

    class Lib:
        @staticmethod
        def tfpa_call(args):
            a = B.tfpa_call_args.from_buffer_copy(args.ljust(ctypes.sizeof(B.tfpa_call_args), b"\0"))
            b.slabs[1] = 7 * FAKE
            b.c()                                              # what the other thread's call does
            junk = [(ctypes.c_void_p * 2)(9 * FAKE, 9 * FAKE) for _ in range(64)]  # noqa: F841
            c = B.tfpa_bounds.from_address(a.bounds)
            seen.append([c.block, c.pool] + [x or 0 for x in (ctypes.c_void_p * 2).from_address(c.slabs)])
            return 0

    monkeypatch.setattr(B, "lib", lambda: Lib)
    for f in (bounds, select):
        b.slabs[1] = FAKE
        f(rows=((1, 5),), b=b, segs=[LONG, SLAB])
    assert seen == [[64, FAKE, 0, FAKE]] * 2


# ---------------------------------------------------------------- element types and sizes
def refuses(what, f):
    """A ValueError that names what is wrong, and no launch."""
    with B.record_launches() as rec, pytest.raises(ValueError) as e:
        f()
    assert what in str(e.value) and not isinstance(e.value, B.TfpaError) and rec == []


def rows_of(n=2, heads=8, dtype=torch.bfloat16):
    return torch.zeros(n, heads, 128, dtype=dtype)


def write(q=None, k=None, v=None, q_out=None, n=2, **kw):
    k = rows_of(n) if k is None else k
    v = rows_of(n) if v is None else v
    B.tfpa_write_qkv(_cache(), [LONG], q, k, v, q_out, [0] * n, list(range(n)), stream=0, **kw)


WRONG_ROWS = [torch.float32, torch.float16, torch.int8, torch.uint8, torch.float64, torch.int32]


@pytest.mark.parametrize("dtype", WRONG_ROWS)
def test_a_projections_rows_are_bf16(dtype):
    """One-byte rows would be read (q_out written) past their end, others are other numbers."""
    bad, q, out = rows_of(dtype=dtype), rows_of(heads=32), rows_of(heads=32)
    refuses("k must", lambda: write(k=bad))
    refuses("v must", lambda: write(v=bad))
    refuses("q must", lambda: write(q=rows_of(heads=32, dtype=dtype), q_out=out))
    refuses("q_out must", lambda: write(q=q, q_out=rows_of(heads=32, dtype=dtype)))


@pytest.mark.parametrize("name", ["q_weight", "k_weight"])
@pytest.mark.parametrize("w", [torch.ones(128, dtype=torch.bfloat16), torch.ones(128, dtype=torch.float16), torch.ones(128, dtype=torch.float64),
                               torch.ones(64), torch.ones(127), torch.ones(8, 128), torch.ones(256)[::2], torch.ones(0)],
                         ids=["bf16", "f16", "f64", "64", "127", "a head each", "strided", "none"])
def test_weights_are_128_float32(name, w):
    """Models hold them as bf16: 256 bytes, where 512 are read."""
    refuses(name, lambda: write(q=rows_of(heads=32), q_out=rows_of(heads=32), **{name: w}))


@pytest.mark.parametrize("pos", [torch.zeros(2), torch.zeros(2, dtype=torch.int64), torch.zeros(2, 2, dtype=torch.int32)[:, 0],
                                 torch.zeros(4, dtype=torch.int32)[::2]], ids=["f32", "i64", "column", "strided"])
def test_rotary_positions_are_int32_one_after_the_other(pos):
    t = torch.zeros(8, 64)
    refuses("rope_pos", lambda: write(rope_cos=t, rope_sin=t, rope_pos=pos))


@pytest.mark.parametrize("dtype", [torch.int32, torch.float16, torch.float64])
def test_tables_are_float32(dtype):
    bad, good = torch.zeros(8, 64, dtype=dtype), torch.zeros(8, 64)
    refuses("rope_cos", lambda: write(rope_cos=bad, rope_sin=good))
    refuses("rope_sin", lambda: write(rope_cos=good, rope_sin=bad))
    refuses("table", lambda: B.tfpa_rope_table(B.RopeSpec(1e4), 0, bad, good, stream=0))
    refuses("table", lambda: B.tfpa_rope_table(B.RopeSpec(1e4), 0, good, bad, stream=0))


def test_tables_come_together():
    """One of the two alone was an AttributeError, or K and q unrotated without a word."""
    t = torch.zeros(8, 64)
    refuses("rope_cos and rope_sin", lambda: write(rope_sin=t))
    refuses("rope_cos and rope_sin", lambda: write(rope_cos=t))


def test_rows_weights_and_tables_that_are_right_are_taken():
    """bf16, or its bits; weights of any shape of 128; addresses."""
    t, w = torch.zeros(8, 64), torch.ones(1, 128)
    with B.record_launches() as rec:
        write(q=rows_of(heads=32), q_out=rows_of(heads=32), q_weight=w, k_weight=w[0], rope_cos=t, rope_sin=t,
              rope_pos=torch.zeros(2, dtype=torch.int32))
        write(k=rows_of(dtype=torch.int16), v=rows_of(dtype=torch.int16))
        write(k_weight=FAKE, rope_cos=t, rope_sin=t, rope_pos=FAKE)
        write(n=0)
    assert [(r["kind"], r["rows"]) for r in rec] == [("write_qkv", 2)] * 3


def lists(n=2, nsel=4):
    return torch.zeros(n, 8, nsel, dtype=torch.int32)


def choose(q, n=2):
    B.tfpa_select_blocks(_cache(), [LONG], B.Bounds(64, FAKE), q, [0] * n, list(range(n)), lists(n), stream=0)


def attend(q, out=FAKE, lse=None, n=2):
    B.tfpa_decode_blocks(_cache(), [LONG], q, [0] * n, list(range(n)), lists(n), 64, 0.1, out, lse, stream=0)


HEADS = rows_of(heads=32)
WRONG_HEADS = {"f32": HEADS.float(), "f16": HEADS.half(), "i8": HEADS.to(torch.int8), "one row": HEADS[:1], "a head less": HEADS[:, :31].contiguous(),
               "strided": rows_of(heads=64)[:, ::2], "rows apart": rows_of(heads=48)[:, :32], "transposed": rows_of(32, 2).transpose(0, 1),
               "none": HEADS[:0]}


@pytest.mark.parametrize("name", WRONG_HEADS)
def test_q_and_out_are_bf16_of_every_row(name):
    """What is smaller than the rows' heads would be read, or written, past its end."""
    bad = WRONG_HEADS[name]
    refuses("q must", lambda: choose(bad))
    refuses("q must", lambda: attend(bad))
    refuses("out must", lambda: attend(HEADS, bad))


@pytest.mark.parametrize("lse", [torch.zeros(2, 32, dtype=torch.bfloat16), torch.zeros(2, 32, dtype=torch.float64), torch.zeros(1, 32),
                                 torch.zeros(2, 31), torch.zeros(2, 64)[:, ::2], torch.zeros(32, 2).t()],
                         ids=["bf16", "f64", "one row", "a head less", "strided", "transposed"])
def test_lse_is_float32_of_every_row(lse):
    refuses("lse must", lambda: attend(HEADS, HEADS, lse))


def test_q_out_and_lse_that_are_right_are_taken():
    """Any shape that holds the rows, buffers for more rows among them; bf16's bits; addresses."""
    with B.record_launches() as rec:
        choose(HEADS)
        choose(HEADS.view(2, -1).view(torch.int16))
        attend(HEADS, HEADS.clone(), torch.zeros(2, 32))
        attend(rows_of(9, 32), rows_of(9, 32).view(-1), torch.zeros(9 * 32))
        attend(FAKE, FAKE, FAKE)
        attend(HEADS[:0], HEADS[:0], torch.zeros(0, 32), n=0)
    assert [r["kind"] for r in rec] == ["select_blocks"] * 2 + ["decode_blocks"] * 3


# ---------------------------------------------------------------- the size of bounds
class Pool:
    """A pool's shape and type without its memory."""

    def __init__(self, *shape, dtype=torch.bfloat16, dense=True, ptr=FAKE):
        self.shape, self.dtype, self._dense, self._p = torch.Size(shape), dtype, dense, ptr

    def is_contiguous(self):
        return self._dense

    def data_ptr(self):
        return self._p


WRONG_POOLS = {"blocks of 128": Pool(4096, 8, 2, 2, 128), "blocks of 256": Pool(4096, 8, 1, 2, 128), "fewer pages": Pool(4095, 8, 4, 2, 128),
               "a head less": Pool(4096, 7, 4, 2, 128), "a head more": Pool(4096, 9, 4, 2, 128), "one bound": Pool(4096, 8, 4, 1, 128),
               "narrow": Pool(4096, 8, 4, 2, 64), "f32": Pool(4096, 8, 4, 2, 128, dtype=torch.float32),
               "i8": Pool(4096, 8, 4, 2, 128, dtype=torch.int8), "strided": Pool(4096, 8, 4, 2, 128, dense=False),
               "flat": Pool(4096 * 8 * 4 * 256)}


@pytest.mark.parametrize("name", WRONG_POOLS)
def test_a_pool_of_bounds_has_the_caches_shape(name):
    """Bounds of 128 positions under blocks of 64 were written past the pool's end."""
    for f in (bounds, select):
        refuses("bounds of", lambda: f(b=B.Bounds(64, WRONG_POOLS[name])))
        refuses("bounds of", lambda: f(b=B.Bounds(64, WRONG_POOLS[name], [None])))


def test_a_pool_is_looked_at_again_for_another_cache_and_another_block():
    b = B.Bounds(64, Pool(4096, 8, 4, 2, 128))
    with B.record_launches() as rec:
        bounds(b=b)
        bounds(b=b)
        bounds(b=B.Bounds(128, Pool(5000, 8, 2, 2, 128, dtype=torch.int16)))
        bounds(b=B.Bounds(64, Pool(4096, 8, 4, 2, 128)), cache=_cache(num_pages=4000))
    assert len(rec) == 4
    refuses("bounds of", lambda: bounds(b=b, cache=_cache(num_pages=4097)))
    refuses("bounds of", lambda: bounds(b=b, cache=_cache(hq=8, hkv=4)))
    b.block = 128
    refuses("bounds of", lambda: bounds(b=b))
    b.block, b.pool = 64, Pool(4096, 8, 2, 2, 128)
    refuses("bounds of", lambda: bounds(b=b))


WRONG_SLABS = {"blocks of 128": Pool(8, 6, 2, 128), "a block less": Pool(8, 11, 2, 128), "a head less": Pool(7, 12, 2, 128),
               "f32": Pool(8, 12, 2, 128, dtype=torch.float32), "strided": Pool(8, 12, 2, 128, dense=False)}


@pytest.mark.parametrize("name", WRONG_SLABS)
@pytest.mark.parametrize("table", [False, True])
def test_bounds_of_a_slab_have_its_shape(name, table):
    """A slab of 768 positions has twelve blocks of 64; heads lie slab_cap / block blocks apart."""
    segs = [LONG, SLAB]
    segs = B.SegTable(segs) if table else segs
    b = B.Bounds(64, FAKE, [None, Pool(8, 12, 2, 128)])
    for f in (bounds, select):
        with B.record_launches() as rec:
            f(rows=((1, 5),), b=b, segs=segs)
        assert len(rec) == 1
        refuses("bounds of", lambda: f(rows=((1, 5),), b=B.Bounds(64, FAKE, [None, WRONG_SLABS[name]]), segs=segs))
    b.slabs[1] = WRONG_SLABS[name]
    refuses("bounds of", lambda: bounds(rows=((1, 5),), b=b, segs=segs))
    longer = B.Seg(700, k_slab=FAKE, v_slab=FAKE, slab_cap=1024)
    refuses("bounds of", lambda: bounds(rows=((1, 5),), b=B.Bounds(64, FAKE, [None, Pool(8, 12, 2, 128)]), segs=[LONG, longer]))


# ---------------------------------------------------------------- launches
@pytest.mark.parametrize("hq,hkv,items", [(32, 8, 64), (64, 8, 64), (72, 8, 64), (128, 8, 64), (256, 8, 128), (16, 1, 8), (128, 1, 64)])
def test_ctas_of_a_batch_are_no_more_than_the_kernel_has_on_the_gpu(hq, hkv, items):
    """Four CTAs a SM with up to eight query heads a kv head, two with more (152 SMs here): eight lists of eight parts."""
    with B.record_launches() as rec:
        B.tfpa_decode_blocks(_cache(hq=hq, hkv=hkv), [LONG], FAKE, [0] * 8, list(range(4000, 4008)), Pool(8, hkv, 64, dtype=torch.int32), 64, 0.1,
                             FAKE, stream=0)
    most = 152 * (4 if hq // hkv <= 8 else 2)
    ctas = max(n for n in (8, 4, 2, 1) if items * n <= most)
    assert [(r["items"], r["grid"]) for r in rec] == [(items, items * ctas)]


def test_launches_of_more_than_64_runs_are_cut():
    """Each launch takes 64 runs; its q, lists and output start at its first row."""
    n, nsel = 150, 5
    rows = [(i % 2, 3 * i) for i in range(n)]
    rs, rp = [r[0] for r in rows], [r[1] for r in rows]
    segs = [LONG, SLAB]
    b = B.Bounds(64, FAKE, [None, 3 * FAKE])
    with B.record_launches() as rec:
        B.tfpa_key_bounds(_cache(), segs, b, rs, rp, stream=0)
        B.tfpa_select_blocks(_cache(), segs, b, FAKE, rs, rp, Pool(n, 8, nsel, dtype=torch.int32), stream=0)
        B.tfpa_decode_blocks(_cache(), segs, FAKE, rs, rp, Pool(n, 8, nsel, dtype=torch.int32), 64, 0.1, FAKE, stream=0)
    cuts = ((0, 64), (64, 64), (128, 22))
    at = [(r["kind"], r["row0"], r["rows"], r["runs"], r["items"], r["q_offset"], r["out_offset"]) for r in rec]
    assert at == ([("key_bounds", a, k, k, 8 * k, 0, 0) for a, k in cuts]
                  + [("select_blocks", a, k, k, 8 * k, a * 32 * 128, a * 8 * nsel) for a, k in cuts]
                  + [("decode_blocks", a, k, k, 8 * k, a * 32 * 128, a * 32 * 128) for a, k in cuts])
