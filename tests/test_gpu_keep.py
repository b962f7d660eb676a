"""tfpa_keep_kv of every number of pairs that its documentation allows, as a process's first calls: what a launch
needs must not depend on a larger call having come before.  Each cache type runs in a process of its own."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
# pairs of a call, ascending: around the counts at which a launch passes 48 KB of shared memory, and the most
COUNTS = {"bf16": [1, 80, 81, 96, 97, 256], "fp8": [160, 161, 192, 193, 256], "fp4": [204, 205, 255, 256]}


def _rows(pool, kv):
    """The pool's stored rows as byte views [pages][hkv][256][...], one or (codes, scales) two."""
    if kv != "fp4":
        return [pool]
    h = pool.unflatten(-1, (2, 9216))
    return [h[..., :8192].unflatten(-1, (128, 64)), h[..., 8192:].unflatten(-1, (128, 8))]


def child(kv):
    import numpy as np
    import torch
    from paged_kv_cache_235_gb300 import binding as B
    hkv, pages = 3, 4
    shape = {"bf16": (256, 256), "fp8": (256, 128), "fp4": (B.FP4_BLOCK,)}[kv]
    torch.manual_seed(1)
    pools = [torch.randint(0, 256, (pages, hkv) + shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    ones, err = torch.ones(hkv, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = B.Cache(kv, hkv, hkv, pools[0], pools[1], ones, ones, err, pages)
    seg = [B.Seg(768, page_table=table)]
    rng = np.random.default_rng(2)
    for n in COUNTS[kv]:
        perm = rng.permutation(768)
        src, dst = perm[:n], rng.permutation(768)[:n]            # overlapping: every source is read first
        want = [p.clone() for p in pools]
        pt = table.long()
        s, d = torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda()
        for p, w in zip(pools, want):
            for a, b in zip(_rows(p, kv), _rows(w, kv)):
                if kv == "fp4":
                    b[pt[d // 256], :, d % 256 // 128, d % 128] = a[pt[s // 256], :, s % 256 // 128, s % 128]
                else:
                    b[pt[d // 256], :, d % 256] = a[pt[s // 256], :, s % 256]
        B.tfpa_keep_kv(cache, seg, np.zeros(n, np.int32), src, dst)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for p, w in zip(pools, want):
            assert torch.equal(p, w), n
    print("kept")


@pytest.mark.parametrize("kv", sorted(COUNTS))
def test_keep_of_as_many_pairs_as_a_call_may_have(kv):
    r = subprocess.run([sys.executable, "-c", f"from tests.test_gpu_keep import child; child({kv!r})"], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "kept" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]
