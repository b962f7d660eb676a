"""Blocks and attention over them on the GPU, at the ends of their definitions: scores that are no numbers, scores that
64 bits cannot tell, weights far below a row's largest, batches of more streams than a launch takes."""

from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests.gpu64 import SCALE, LongCase, last_rows
from tests.test_gpu_blocks import (KVS, attend64, blocks_of, bound_store, bound_view, check_choice, exact_bounds, one,
                                   random_bounds, random_lists, run_attend)

pytestmark = pytest.mark.gpu


def selected(c, b, q, rs, rp, nsel, sink=0, recent=0):
    got = torch.empty(len(rs), c.hkv, nsel, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, got, sink=sink, recent=recent)
    return got.cpu().numpy()


# ---------------------------------------------------------------- selection
@pytest.mark.parametrize("L", [3000, 20000])               # few blocks too near to tell, and many
def test_a_score_that_is_no_number_counts_as_largest(L):
    """NaN (0 times an infinite bound) before +inf, and of each the lower block first."""
    c, b, rs, rp = one(L)
    q = c.q(1).abs()
    q[..., 4] = 0.0
    at = blocks_of(c, b)
    for blk, dim in ((5, 9), (11, 4), (17, 9), (20, 4), (31, 9)):      # dim 9: +inf; dim 4, under zeros of q: NaN
        b.pool[at[blk][0], :, at[blk][1], 1, dim] = float("inf")
    for nsel, want in ((1, [11]), (2, [11, 20]), (3, [5, 11, 20]), (4, [5, 11, 17, 20]), (5, [5, 11, 17, 20, 31])):
        assert selected(c, b, q, rs, rp, nsel)[0, 0].tolist() == want


@pytest.mark.parametrize("n", [47, 200])
def test_scores_that_64_bits_cannot_tell(n):
    """Large bounds that cancel: a chosen block's exact score is below another's by no more than the two sums' roundings."""
    c = LongCase("bf16", [64 * n], [True], 1, 1, 201)
    b = bound_store(c, 64)
    b.pool.zero_()
    rng = np.random.default_rng(n)
    at = blocks_of(c, b)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device="cuda")
    q[..., :8] = 1.0
    e = np.zeros((n, 8))
    for i in range(n):
        big = 2.0 ** rng.integers(40, 62)
        e[i] = rng.permutation([big, -big, 2 * big, -2 * big, *(rng.integers(1, 9, 4) / 8.0)])
        b.pool[at[i][0], 0, at[i][1], 1, :8] = torch.from_numpy(e[i]).to(torch.bfloat16)
    exact = [sum(Fraction(float(x)) for x in row) for row in e]
    off = [(14 + 1) * Fraction(1, 2 ** 53) * sum(abs(Fraction(float(x))) for x in row) for row in e]
    for nsel in (1, 10, 40):
        got = selected(c, b, q, [0], [64 * n - 1], nsel)[0, 0]
        assert (got >= 0).all() and (np.diff(got) > 0).all()
        assert np.array_equal(got, selected(c, b, q, [0], [64 * n - 1], nsel)[0, 0])
        rest = sorted(set(range(n)) - set(got.tolist()))
        assert all(exact[i] >= exact[j] - off[i] - off[j] for i in got for j in rest)


def many(seed, L0=1000):
    """Seventy-odd streams, paged and in slabs, most with one row."""
    rng = np.random.default_rng(seed)
    lengths = [int(x) for x in rng.integers(L0, 6 * L0, 75)]
    return lengths, [i % 4 != 2 for i in range(75)]


@pytest.mark.parametrize("single", [True, False])
def test_more_streams_than_a_launch_takes(single):
    """Bounds, blocks and attention of 75 runs: the second launch's rows, bounds, q and lists are its own."""
    lengths, paged = many(202)
    c = LongCase("fp8", lengths, paged, 8, 2, 203)
    b = bound_store(c, 64)
    counts = [1 if single else 1 + (i % 7 == 3) * (i % 4) for i in range(75)]
    rs, rp = last_rows(lengths, counts)
    B.tfpa_key_bounds(c.cache, c.segs, b, rs, rp)
    for s, (L, n) in enumerate(zip(lengths, counts)):
        touched = set(range((L - n) // 64, (L - 1) // 64 + 1))
        for blk in touched:
            assert torch.allclose(bound_view(c, b, s, blk).double(), exact_bounds(c, s, blk, 64), rtol=1e-7, atol=0), (s, blk)
        before = min(touched) - 1
        assert (bound_view(c, b, s, before) == 3.0).all(), s
    b = random_bounds(c, 64, 204)
    q = c.q(len(rs))
    lists = torch.full((len(rs) + 2, 2, 9), 77, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists[1:-1], sink=1, recent=2)
    assert (lists[[0, -1]] == 77).all()
    check_choice(c, b, q, rs, rp, 9, 1, 2, got=lists[1:-1])
    lists = lists[1:-1].contiguous()
    out, lse = run_attend(c, q, rs, rp, lists, 64)
    ref, rl, tol, ltol = attend64(c, q, rs, rp, lists, 64)
    assert ((out.double() - ref).abs() <= tol).all() and ((lse.double() - rl).abs() <= ltol).all()
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("streams,L", [(160, 9000), (70, 40000)])
def test_a_batch_in_which_one_cta_chooses_for_a_row(streams, L):
    """So many rows that a cluster is one CTA: hundreds of blocks each, named by tables that share their pages."""
    c = LongCase("bf16", [8192], [True], 32, 8, 205)
    b = random_bounds(c, 64, 206)
    rng = np.random.default_rng(207)
    c.lengths = [int(x) for x in rng.integers(L // 2, L, streams)]
    c.segs = [B.Seg(n, page_table=torch.from_numpy(rng.integers(0, c.num_pages, -(-n // 256)).astype(np.int32)).cuda()) for n in c.lengths]
    rs, rp = last_rows(c.lengths, [1] * streams)
    q = c.q(streams)
    with B.record_launches() as rec:
        B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, torch.empty(streams, 8, 20, dtype=torch.int32, device="cuda"), stream=0)
    assert [r["grid"] // r["items"] for r in rec][0] == 1                 # the full launch of 64 rows: 512 items
    got = torch.empty(streams, 8, 20, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, got, sink=1, recent=2)
    pick = np.array([0, 1, 33, 62, 63, 64, 65, streams - 1])
    at = torch.from_numpy(pick).cuda()
    check_choice(c, b, q[at].contiguous(), rs[pick], rp[pick], 20, 1, 2, got=got[at])


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("nsel", [2, 16, 64])
def test_weights_far_below_a_rows_largest(kv, nsel):
    """A sixteenth of the keys takes nearly all the weight and has no value: what comes out is the sum of weights of
    2^-20 to 2^-28 of the largest."""
    c = LongCase(kv, [4096], [True], 4, 1, 208)
    k, v = torch.zeros(4096, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(4096, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[::16, :, 0], v[::16] = 4.0, 0.0
    v[:, :, 64:] *= -0.5
    B.tfpa_write_kv(c.cache, c.segs, k, v, np.zeros(4096), np.arange(4096))
    k0 = float(c.values(0, 0, 0)[0, 0])                # 4 as it is stored
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    q[0, :, 0] = torch.tensor([20.0, 24.0, 26.0, 28.0], device="cuda") * float(np.log(2)) / (SCALE * k0)
    lists = random_lists(c, [0], [4095], nsel, 64, 209)
    out, lse = run_attend(c, q, [0], [4095], lists, 64)
    ref, rl, tol, ltol = attend64(c, q, [0], [4095], lists, 64)
    # tol has an absolute part of 2^-25 of the largest weight a key, which would let all of these go; here a key's
    # weight may be off by 2^-32 of the largest (f16's last bit, 2^-24, halved, of weights up to 2^7)
    K, V = c.values(0, 0, 0), c.values(0, 1, 0)
    key = (lists[0, 0].long()[:, None] * 64 + torch.arange(64, device="cuda")).flatten()
    e = (SCALE * q[0].double() @ K[key].T)
    e = (e - e.amax(-1, keepdim=True)).exp()
    z = e.sum(-1, keepdim=True)
    es = 2 * 128 * 2.0 ** -24 * 28 * float(np.log(2)) + 2.0 ** -20           # of a score, as attend64 has it
    small = 2.0 ** -8 * ref[0].abs() + (e @ V[key].abs() / z) * (2.0 ** -11 + 2 * es) + len(key) * 2.0 ** -32 / z * V.abs().max()
    err = (out[0].double() - ref[0]).abs()
    assert (ref[0].abs() > 4 * small).all()            # the test tells them from nothing
    assert (err <= small).all(), (err / small).max()
    assert ((lse.double() - rl).abs() <= ltol).all()
