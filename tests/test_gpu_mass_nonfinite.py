"""The attention weight beside values that are not finite: columns that no row of the call fills, rows that saw no
key, and rows whose query is not a number must leave the keys that are not theirs alone."""

import numpy as np
import pytest
import torch

from tests import fp4_cases as F
from tests.test_gpu_evict import make, mass64, run_mass

pytestmark = pytest.mark.gpu

F32_MIN_NORMAL = 2.0 ** -126


def _set_bf16_key(c, seg, pos, dim, bits):
    """Key `pos` of every kv head of a paged bf16 stream, on both sides."""
    pid = int(seg.page_table[pos // 256])
    c.cache.k_pool[pid, :, pos % 256, dim] = bits
    c.k_pool.view(torch.int16)[pid, :, pos % 256, dim] = int(np.array(bits, np.uint16).view(np.int16))


@pytest.mark.parametrize("hq,hkv,rows", [(8, 2, 1), (3, 3, 1), (20, 4, 3)])
def test_mass_of_an_infinite_key(hq, hkv, rows):
    """A key element of -inf under queries that are positive there: a score of -inf, so a weight of 0.  The call's
    vectors fill 4, 1 and 15 of a product's 16 columns; what stands in the others is no row's weight."""
    c = make("bf16", [300], [True], hq, hkv, seed=91)
    key, dim = 10, 5
    _set_bf16_key(c, c.segs[0], key, dim, 0xFF80)
    q = c.q(rows)
    q[..., dim] = F.bf16_bits(np.full(q.shape[:2], 0.75))
    lse = np.full((rows, hq), 4.0, np.float32)
    rs, rp = np.zeros(rows, int), np.arange(300 - rows, 300)
    m = run_mass(c, q, lse, rs, rp, np.zeros((1, hkv, 304), np.float32), 0.0).cpu().numpy().astype(np.float64)
    assert np.isfinite(m).all() and (m[0, :, key] == 0).all()
    _set_bf16_key(c, c.segs[0], key, dim, 0)                      # the other keys: the plain sums
    ref, tol = mass64(c, q, lse, rs, rp, np.zeros((1, hkv, 304), np.float32), 0.0, 304)
    ref[0, :, key] = 0
    F.assert_within(m, ref, tol + 1e-300, "other keys")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80, 0x7E00])
@pytest.mark.parametrize("none", [0, 1])
def test_mass_of_rows_that_saw_no_key_whatever_their_query_holds(kv, bits, none):
    """lse = -inf adds nothing: the same bytes with a query of NaN, of infinity or of 2^125 in that row as with
    zeros, for the call's other rows too."""
    c = make(kv, [400], [True], 8, 2, seed=92)
    q, lse = c.q(3), np.full((3, 8), 4.0, np.float32)
    lse[none] = -np.inf
    rs, rp = np.zeros(3, int), np.array([397, 398, 399])
    old = np.ones((1, 2, 400), np.float32)
    q[none] = 0
    want = run_mass(c, q, lse, rs, rp, old, 0.5)
    q[none] = bits
    got = run_mass(c, q, lse, rs, rp, old, 0.5)
    assert torch.isfinite(want).all() and torch.equal(got, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("bits", [0x7FC0, 0x7F80])
def test_mass_of_a_query_that_is_not_finite_stays_with_its_keys(kv, bits):
    """A row at position 100 whose query is not finite spoils keys 0 to 100 at most: the keys behind it keep the
    later row's weights."""
    c = make(kv, [400], [True], 8, 2, seed=93)
    q, lse = c.q(2, 8.0), np.full((2, 8), 30.0, np.float32)
    rs, rp = np.zeros(2, int), np.array([100, 399])
    old = np.zeros((1, 2, 400), np.float32)
    q[0, :, 3] = bits
    got = run_mass(c, q, lse, rs, rp, old, 0.0).cpu().numpy().astype(np.float64)
    ref, tol = mass64(c, q[1:], lse[1:], rs[1:], rp[1:], old, 0.0, 400)
    F.assert_within(got[..., 101:], ref[..., 101:], tol[..., 101:] + F32_MIN_NORMAL, "keys behind the row")
