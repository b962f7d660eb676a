"""Eviction with positions of the slots' own: which keys count as the first and the last ones when the call gives
no next_pos, and when a slot's position has not been written.  Against a sort in 64 bits."""

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests.fp4_cases import Fp4Case, dev
from tests.test_gpu_evict import masses

pytestmark = pytest.mark.gpu


def want(mass, pos, L, n, sink, recent):
    """Slots that fill the first n, of one kv head; the last positions are those up to the largest that is held."""
    m, p = mass[:L].astype(np.float64), pos[:L]
    guard = ((p >= 0) & (p < sink)) | (p >= p.max() + 1 - recent)
    stays = np.zeros(L, bool)
    stays[np.lexsort((np.arange(L), -m, ~guard))[:n]] = True
    take = np.arange(n)
    take[~stays[:n]] = np.flatnonzero(stays[n:]) + n
    return take


def check(c, keep, mass, pos, sink, recent):
    dm, dp, mv = dev(mass), dev(pos), B.make_moves(len(c.lengths), c.hkv, mass.shape[2])
    B.tfpa_evict_kv(c.gcache, c.gsegs, keep, dm, mv, key_pos=dp, sink=sink, recent=recent)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    gm, gp = dm.cpu().numpy(), dp.cpu().numpy()
    for s, L in enumerate(c.lengths):
        n = int(keep[s])
        for g in range(c.hkv):
            take = want(mass[s, g], pos[s, g], L, n, sink, recent)
            assert np.array_equal(gp[s, g, :n], pos[s, g, take]) and np.array_equal(gm[s, g, :n], mass[s, g, take]), (s, g)
            assert (gp[s, g, n:L] == -1).all() and (gm[s, g, n:L] == 0).all()
    return gp


@pytest.mark.parametrize("lengths", [[600, 333], [20000], [60001, 5]])
def test_a_later_cut_without_next_pos(lengths):
    """What earlier cuts left: positions far past the number of slots.  The last `recent` are counted from the
    largest position that a head holds, and the weights choose among the rest."""
    c = Fp4Case(lengths, [True, False][: len(lengths)], 4, 2, seed=95).upload()
    rng = np.random.default_rng(3)
    mass = masses(c, 5)
    pos = np.full(mass.shape, -1, np.int32)
    for s, L in enumerate(lengths):
        for g in range(2):
            pos[s, g, :L] = rng.permutation(np.sort(rng.choice(4 * L, L, replace=False)))
    keep = np.array([max(4, L // 2) for L in lengths], np.int32)
    check(c, keep, mass, pos, sink=2, recent=2)


@pytest.mark.parametrize("sink,recent", [(4, 0), (4, 16), (0, 1)])
def test_slots_without_a_position_are_not_protected(sink, recent):
    """-1: a row whose entry the caller has not written yet.  Its weight alone decides."""
    c = Fp4Case([500], [True], 4, 2, seed=96).upload()
    mass = masses(c, 6)
    pos = np.broadcast_to(np.arange(mass.shape[2], dtype=np.int32), mass.shape).copy()
    pos[:, :, 200:230] = -1
    mass[:, :, 200:215] = 0                                      # goes
    mass[:, :, 215:230] = 1e6                                    # stays
    gp = check(c, np.array([250], np.int32), mass, pos, sink, recent)
    assert (np.count_nonzero(gp[0, :, :250] == -1, axis=1) == 15).all()
