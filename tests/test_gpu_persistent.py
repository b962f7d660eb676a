"""The persistent kernels where every CTA has several work items: rings, tensor-memory buffers and barriers that come
round again, items that go on from one another, key tiles by the dozen.  Against 64 bits on the GPU, and a
stream's bytes in a batch against its bytes alone, where its items are no more than the SMs."""

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests import gpu64 as X

pytestmark = pytest.mark.gpu

LENGTHS = [15000, 20001, 16385, 18111, 17408, 19999, 16640, 15873]


def _case(kv="fp4", lengths=LENGTHS, hq=32, hkv=8, seed=1):
    return X.LongCase(kv, lengths, [i % 2 == 0 for i in range(len(lengths))], hq, hkv, seed)


def _items(c, rs, rp, kind="partial"):
    """Work items of each launch of a call, from a dry run."""
    with B.record_launches() as rec:
        B.tfpa_decode(c.cache, c.segs, 1 << 20, rs, rp, X.SCALE, B.Scratch(1 << 20, 1 << 21, 1 << 16, 32), 1 << 22, None, stream=0)
    return [r["items"] for r in rec if r["kind"] == kind]


def _decode(c, q, rs, rp, anc=None, rows=None):
    """A call over the rows (of `rows` only), with scratch for all of them."""
    at = np.arange(len(rs)) if rows is None else rows
    q, rs, rp = q[torch.from_numpy(at).cuda()].contiguous(), rs[at], rp[at]
    out = torch.empty(len(at), c.hq, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(len(at), c.hq, device="cuda")
    sc = B.make_scratch(len(at), c.hq)
    if anc is None:
        B.tfpa_decode(c.cache, c.segs, q, rs, rp, X.SCALE, sc, out, lse)
    else:
        B.tfpa_decode_tree(c.cache, c.segs, q, rs, rp, anc[torch.from_numpy(at).cuda()].contiguous(), X.SCALE, sc, out, lse)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    return out, lse


def _check(c, counts, anc=None, what=""):
    rs, rp = X.last_rows(c.lengths, counts)
    q = c.q(len(rs))
    out, lse = _decode(c, q, rs, rp, anc)
    ref, rl, tol, lt = X.attend(c, q, rs, rp, anc)
    X.assert_within(out, ref, tol, what + " out")
    X.assert_within(lse, rl, lt, what + " lse")
    for s in range(len(c.lengths)):              # the same bytes alone
        at = np.flatnonzero(rs == s)
        if len(at):
            o, l = _decode(c, q, rs, rp, anc, at)
            at = torch.from_numpy(at).cuda()
            assert torch.equal(o, out[at]) and torch.equal(l, lse[at]), (what, s)
    return rs, rp, q, out, lse


@pytest.mark.parametrize("rows", [1, 2, 3, 4])
def test_decode_over_4_bits(rows):
    """4, 8, 12 and 16 vectors a kv head: the kernel of eight-vector items and the one of sixteen."""
    c = _case(seed=100 + rows)
    rs, rp = X.last_rows(c.lengths, [rows] * 8)
    assert min(_items(c, rs, rp)) > 6 * 152
    _check(c, [rows] * 8, what=f"rows {rows}")


def test_decode_over_4_bits_both_kernels_in_a_call():
    c = _case(seed=105)
    counts = [1, 4, 2, 3, 1, 4, 2, 3]
    rs, rp = X.last_rows(c.lengths, counts)
    items = _items(c, rs, rp)
    assert len(items) == 2 and min(items) > 2 * 152
    _check(c, counts, what="mixed")


@pytest.mark.parametrize("hq,hkv,n", [(8, 1, 32), (10, 2, 16), (6, 2, 16)])
def test_decode_over_4_bits_of_few_kv_heads(hq, hkv, n):
    """Fewer than eight kv heads: splits of two pages, items of few stages, groups of 8, 5 and 3."""
    c = _case(lengths=[14000 + 331 * i for i in range(n)], hq=hq, hkv=hkv, seed=106 + hkv)
    rs, rp = X.last_rows(c.lengths, [1] * n)
    assert max(_items(c, rs, rp)) > 4 * 152      # (a launch takes 15 slabs)
    _check(c, [1] * n, what=f"{hq}/{hkv}")


@pytest.mark.parametrize("rows", [2, 4])
def test_tree_rows_over_4_bits(rows):
    c = _case(seed=110 + rows)
    rng = np.random.default_rng(rows)
    masks = []
    for _ in range(8):
        par = [-1] + [int(rng.integers(0, i)) for i in range(1, rows)]
        for i in range(rows):
            m, a = ((1 << 64) - 1) & ~((1 << (i + 1)) - 1), i
            while a >= 0:
                m, a = m | 1 << (i - a), par[a]
            masks.append(m)
    anc = torch.from_numpy(np.array(masks, np.uint64).view(np.int64)).cuda()
    _check(c, [rows] * 8, anc, f"tree {rows}")


@pytest.mark.parametrize("rows", [1, 2, 4])
def test_append_over_4_bits(rows):
    """A step that stores its rows: the bytes of a store and a decode."""
    a, b = (_case(seed=120) for _ in range(2))
    rs, rp = X.last_rows(a.lengths, [rows] * 8)
    q = a.q(len(rs))
    k, v = (torch.randn(len(rs), 8, 128, generator=a.g, device="cuda").to(torch.bfloat16) for _ in range(2))
    sc = B.make_scratch(len(rs), 32)
    outs = [(torch.empty(len(rs), 32, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(len(rs), 32, device="cuda")) for _ in range(2)]
    B.tfpa_decode_append(a.cache, a.segs, k, v, q, rs, rp, X.SCALE, sc, *outs[0])
    B.tfpa_write_kv(b.cache, b.segs, k, v, rs, rp)
    B.tfpa_decode(b.cache, b.segs, q, rs, rp, X.SCALE, sc, *outs[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)
    for s in a.slabs:
        assert torch.equal(a.slabs[s][0], b.slabs[s][0]) and torch.equal(a.slabs[s][1], b.slabs[s][1])
    ref, rl, tol, lt = X.attend(b, q, rs, rp)
    X.assert_within(outs[0][0], ref, tol, "out")
    X.assert_within(outs[0][1], rl, lt, "lse")


def test_merge_in_the_kernel_over_4_bits():
    """Streams of up to four splits, many of them: the combiners merge item after item."""
    L = [900 + i for i in range(96)]
    c = _case(lengths=L, seed=130)
    rs, rp = X.last_rows(L, [1] * 96)
    assert max(_items(c, rs, rp)) > 4 * 152
    q = c.q(96)
    out, lse = _decode(c, q, rs, rp)
    sc = B.make_scratch(96, 32, fused_merge=True)
    for _ in range(3):
        o, l = torch.empty_like(out), torch.empty_like(lse)
        B.tfpa_decode(c.cache, c.segs, q, rs, rp, X.SCALE, sc, o, l)
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(l, lse) and int(sc.arrive.count_nonzero()) == 0
    ref, rl, tol, lt = X.attend(c, q, rs, rp)
    X.assert_within(out, ref, tol, "out")
    X.assert_within(lse, rl, lt, "lse")


# rows: vectors of a kv head in one product of 16 columns; the epilogue's two tiles at a time; two passes over the
# keys, two buffers of 256 columns
@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("rows", [1, 8, 32, 70])
@pytest.mark.parametrize("decay", [0.0, 0.75])
def test_mass_of_dozens_of_tiles_a_cta(kv, rows, decay):
    """2 streams of 8 kv heads of 300 and 257 key tiles: 29 a CTA, a ring of four or eight stages, tiles and CTAs that end
    inside a head."""
    L = [38401, 32896]
    c = _case(kv, L, seed=140 + rows)
    rs, rp = X.last_rows(L, [rows, rows])
    q = c.q(2 * rows)
    lse = torch.randn(2 * rows, 32, generator=c.g, device="cuda").abs() + 8
    old = torch.rand(2, 8, 38404, generator=c.g, device="cuda")
    m = old.clone()
    B.tfpa_key_mass(c.cache, c.segs, q, lse, rs, rp, X.SCALE, m, decay=decay)
    torch.cuda.synchronize()
    ref, tol = X.mass(c, q, lse, rs, rp, old, decay)
    X.assert_within(m, ref, tol, f"{kv} {rows}")
    m2 = old.clone()
    B.tfpa_key_mass(c.cache, c.segs, q, lse, rs, rp, X.SCALE, m2, decay=decay)
    assert torch.equal(m, m2) and int(c.err.item()) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_more_heads_a_kv_head_than_a_tile_holds(kv):
    """160 query heads on one kv head: ten m-tiles a split, a row's own."""
    L = [3001 + 517 * i for i in range(12)]
    c = _case(kv, L, hq=160, hkv=1, seed=150)
    rs, rp = X.last_rows(L, [1] * 12)
    assert max(_items(c, rs, rp)) > 4 * 152
    q = c.q(12)
    out, lse = _decode(c, q, rs, rp)
    ref, rl, tol, lt = X.attend(c, q, rs, rp)
    if kv == "bf16":                             # the weights are rounded to bf16 there: 2^-8 of each, not 2^-11
        tol = 8 * tol
    X.assert_within(out, ref, tol, "out")
    X.assert_within(lse, rl, lt, "lse")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_mass_of_more_heads_than_a_pass_holds(kv):
    """300 query heads on one kv head, three rows: passes of 256 vectors that begin inside a row."""
    L = [20001, 3000]
    c = _case(kv, L, hq=300, hkv=1, seed=151)
    rs, rp = X.last_rows(L, [3, 2])
    q = c.q(5)
    lse = torch.randn(5, 300, generator=c.g, device="cuda").abs() + 8
    m = torch.zeros(2, 1, 20001, device="cuda")
    B.tfpa_key_mass(c.cache, c.segs, q, lse, rs, rp, X.SCALE, m, decay=0.0)
    torch.cuda.synchronize()
    ref, tol = X.mass(c, q, lse, rs, rp, torch.zeros_like(m), 0.0)
    X.assert_within(m, ref, tol, kv)
