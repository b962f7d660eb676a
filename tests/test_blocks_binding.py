"""Host-side tests of what the Python calls from the projection to attention over selected blocks hand to the
library, and of what they refuse before they call it (no GPU)."""

import ctypes

from paged_kv_cache_235_gb300 import binding as B
from tests.test_blocks_host import FAKE, LONG, SLAB, bounds, select


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
