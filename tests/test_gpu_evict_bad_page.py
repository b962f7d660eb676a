"""Eviction beside a page id that is out of range: the pairs that leave their rows leave what is kept per slot."""

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests.fp4_cases import dev
from tests.test_gpu_evict import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("bad_page", [0, 2])
@pytest.mark.parametrize("bad_id", [-5, 9999])
def test_weight_and_position_stay_with_the_row(kv, bad_page, bad_id):
    """Movers on page 2 and on page 1, holes on page 0.  With page 2 bad its movers stay; with page 0 bad all do."""
    L, n, cap = 700, 110, 704
    c = make(kv, [L], [True], 2, 2, seed=97)
    t = c.gsegs[0].page_table.clone()
    t[bad_page] = bad_id
    mass, pos = np.zeros((1, 2, cap), np.float32), np.full((1, 2, cap), -1, np.int32)
    pos[0, :, :L] = np.arange(L)
    mass[0, :, 300:400] = np.arange(1, 101)                      # kept, from a good page
    mass[0, :, 600:610] = 200                                    # kept, from page 2
    before, dm, dp, mv = c.k_pool.clone(), dev(mass), dev(pos), B.make_moves(1, 2, cap)
    B.tfpa_evict_kv(c.gcache, [B.Seg(L, page_table=t)], [n], dm, mv, key_pos=dp)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 1
    c.err.zero_()
    src = np.r_[300:400, 600:610]
    gm, gp, pairs = dm.cpu().numpy()[0], dp.cpu().numpy()[0], mv.cpu().numpy()[0]
    for g in range(2):
        assert pairs[g, 0] == n and np.array_equal(pairs[g, 4:4 + 2 * n].reshape(-1, 2), np.stack([src, np.arange(n)], 1))
    moved = np.zeros(n, bool) if bad_page == 0 else src < 512
    m, p = mass[0, 0].copy(), pos[0, 0].copy()
    m[n:L], p[n:L] = 0, -1                                       # evicted behind the cut
    for i in range(n):
        if moved[i]:
            m[i], p[i] = mass[0, 0, src[i]], src[i]
        else:                                                    # both slots as they were
            m[src[i]], p[src[i]] = mass[0, 0, src[i]], src[i]
    for g in range(2):
        assert np.array_equal(gm[g], m) and np.array_equal(gp[g], p)
    if bad_page == 0:
        assert torch.equal(c.k_pool, before)
