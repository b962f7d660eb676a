"""Accumulated attention weight and eviction by it, on the GPU against plain forms in 64 bits."""

import numpy as np
import pytest
import torch

from oracle import fp4, kvcache
from paged_kv_cache_235_gb300 import binding as B
from paged_kv_cache_235_gb300 import workloads as wl
from tests import fp4_cases as F
from tests.fp4_cases import SCALE, dev, dev_bf16

pytestmark = pytest.mark.gpu


def make(kv, lengths, paged, hq=8, hkv=2, seed=1):
    """A cache of any type with .cache / .segs (oracle) and .gcache / .gsegs, .q, .err."""
    if kv == "fp4":
        return F.Fp4Case(lengths, paged, hq, hkv, seed).fill().upload()
    from tests.gpu_cases import GpuCase, fp8_scales
    from tests.oracle_cases import build_oracle_cache
    npages = sum((L + 255) // 256 for L, p in zip(lengths, paged) if p) + 2
    tables = wl.permuted_tables(list(lengths), list(paged), npages, seed)
    streams = [wl.Stream(L, p, t, 0 if p else ((L + 255) // 256) * 256) for L, p, t in zip(lengths, paged, tables)]
    w = wl.Workload(f"evict{seed}", hq, hkv, kv, npages, streams, np.zeros(1, np.int32), np.zeros(1, np.int32), seed)
    scales = fp8_scales(w) if kv == "fp8" else None
    c = GpuCase(w, scales)
    c.gcache, c.gsegs, c.hq, c.hkv, c.lengths = c.cache, c.segs, hq, hkv, list(lengths)
    c.cache, c.segs = build_oracle_cache(w, *(scales or (None, None)))
    c.num_pages = npages
    rng = np.random.default_rng(seed)
    c.q = lambda rows, scale=1.0: F.bf16_bits(rng.standard_normal((rows, hq, 128)) * scale)
    return c


def mass64(c, q, lse, rs, rp, old, decay, cap):
    """The sums and what the kernel's roundings allow: a weight's exponent is off by the float32 rounding of
    128 products' sum (128 2^-24 sum |q k| scale, twice for the order) and of score and lse (2^-23 of
    their magnitudes), and by 2^-20 for the exponential; the sums round at every addition (2^-24 each)."""
    out, tol = old.astype(np.float64).copy(), np.zeros(old.shape)
    qf = kvcache.bf16_to_f64(q)
    G = c.hq // c.hkv
    for s in sorted(set(int(x) for x in rs)):
        L = c.lengths[s]
        for g in range(c.hkv):
            K, _ = kvcache.gather(c.cache, c.segs[s], g, L)
            add, err = np.zeros(L), np.zeros(L)
            rows = [r for r in range(len(rs)) if rs[r] == s]
            for r in rows:
                for h in range(g * G, (g + 1) * G):
                    if np.isneginf(lse[r, h]):
                        continue
                    x = SCALE * (K @ qf[r, h])
                    xa = SCALE * (np.abs(K) @ np.abs(qf[r, h]))
                    w = np.where(np.arange(L) <= rp[r], np.exp(np.minimum(x - np.float64(lse[r, h]), 80)), 0)
                    add += w
                    err += w * (2 * 128 * 2.0 ** -24 * xa + 2.0 ** -23 * (np.abs(x) + abs(lse[r, h])) * 2 + 2.0 ** -20)
            n = len(rows) * G + 2
            out[s, g, :L] = (decay * old[s, g, :L] if decay else 0) + add
            tol[s, g, :L] = err + n * 2.0 ** -24 * (add + np.abs(out[s, g, :L])) + 1e-37
    return out, tol


def run_mass(c, q, lse, rs, rp, old, decay, segs=None):
    m = dev(old)
    B.tfpa_key_mass(c.gcache, segs or c.gsegs, dev_bf16(q), dev(lse), rs, rp, SCALE, m, decay=decay)
    torch.cuda.synchronize()
    return m


def check_mass(c, rs, rp, decay, what="", seed=0):
    rng = np.random.default_rng(seed)
    rs, rp = np.asarray(rs), np.asarray(rp)
    q = c.q(len(rs))
    _, lse, _, _ = F.attend64(c.cache, c.segs, q, rs, rp, SCALE)
    lse = lse.astype(np.float32)
    cap = (max(c.lengths) + 259) // 4 * 4
    old = rng.random((len(c.lengths), c.hkv, cap)).astype(np.float32)
    m = run_mass(c, q, lse, rs, rp, old, decay)
    got = m.cpu().numpy().astype(np.float64)
    ref, tol = mass64(c, q, lse, rs, rp, old, decay, cap)
    F.assert_within(got, ref, tol + 1e-300, what)
    assert torch.equal(m, run_mass(c, q, lse, rs, rp, old, decay))         # the same bytes again
    assert int(c.err.item()) == 0
    return ref


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (5, 1), (32, 8), (20, 1)])
def test_mass_of_decode_rows(kv, hq, hkv):
    c = make(kv, [700, 300, 1], [True, False, True], hq, hkv, seed=51)
    check_mass(c, [0, 1, 2], [699, 299, 0], 1.0, f"{kv} {hq}/{hkv}")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("L", [1, 31, 32, 33, 127, 128, 129, 256, 257, 511])
def test_mass_lengths_around_tile_edges(kv, L):
    c = make(kv, [L, L], [True, False], seed=52)
    check_mass(c, [0, 1], [L - 1, L - 1], 0.5, f"{kv} L={L}")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("R", [2, 7, 16, 17, 33, 70, 200])
def test_mass_of_windows(kv, R):
    """The last R rows: more query vectors than are staged at once, and the causal edge inside the window."""
    L = [600, 333]
    c = make(kv, L, [True, False], 8, 2, seed=53)
    rs, rp = wl.decode_rows(L, R)
    check_mass(c, rs, rp, 0.9, f"{kv} R={R}")


def test_a_row_gives_one_per_head():
    c = make("bf16", [900], [True], 8, 2, seed=54)
    q = c.q(5)
    rs, rp = np.zeros(5, int), np.arange(895, 900)
    sc = B.make_scratch(8, 8)
    out, lse = torch.empty(5, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 8, device="cuda")
    B.tfpa_decode(c.gcache, c.gsegs, dev_bf16(q), rs, rp, SCALE, sc, out, lse)
    m = torch.zeros(1, 2, 1024, device="cuda")
    B.tfpa_key_mass(c.gcache, c.gsegs, dev_bf16(q), lse, rs, rp, SCALE, m)
    assert (m.sum(-1) - 20).abs().max() < 1e-3 and (m[..., 900:] == 0).all() and (m >= 0).all()


@pytest.mark.parametrize("decay", [0.0, 0.25, 1.0])
def test_mass_rows_in_any_order_and_many_runs(decay):
    """Rows of three streams mixed, repeated and more runs than a launch holds: decay counts once."""
    c = make("fp4", [500, 257, 64], [True, False, True], 4, 2, seed=55)
    rng = np.random.default_rng(2)
    rs = rng.integers(0, 2, 150)
    rp = np.array([rng.integers(0, c.lengths[s]) for s in rs])
    rs[:70], rp[:70] = 0, np.arange(0, 140, 2)
    ref = check_mass(c, rs, rp, decay, "mixed")
    assert ref.shape[0] == 3


def test_mass_leaves_what_it_does_not_own():
    """Entries past seq_len, and segments without rows; with decay 0 the old sums may be NaN."""
    c = make("bf16", [300, 200], [True, True], seed=56)
    q, lse = c.q(1), np.zeros((1, 8), np.float32)
    old = np.full((2, 2, 512), np.nan, np.float32)
    m = run_mass(c, q, lse, [0], [299], old, 0.0)
    assert torch.isfinite(m[0, :, :300]).all() and torch.isnan(m[0, :, 300:]).all() and torch.isnan(m[1]).all()
    lse[:] = -np.inf                                         # a row that saw no key
    m = run_mass(c, q, lse, [0], [299], np.ones((2, 2, 512), np.float32), 1.0)
    assert (m == 1).all()


def test_mass_ignores_unwritten_keys():
    c = F.Fp4Case([600], [True], seed=57).fill()
    for g in range(2):
        fp4.set_rows(c.cache, c.segs[0], "k", g, np.arange(301, 600), np.full((299, 64), 0x77, np.uint8),
                     np.full((299, 8), 0x7F, np.uint8))
    c.upload()
    q, lse = c.q(1), np.zeros((1, 8), np.float32)
    m = run_mass(c, q, lse, [0], [300], np.zeros((1, 2, 600), np.float32), 1.0)
    assert torch.isfinite(m).all() and (m[..., 301:] == 0).all() and (m[..., :301] > 0).all()


def test_mass_bad_page():
    c = make("fp8", [700], [True], seed=58)
    t = c.gsegs[0].page_table.clone()
    t[1] = 9999
    q, lse = c.q(1), np.zeros((1, 8), np.float32)
    m = run_mass(c, q, lse, [0], [699], np.ones((1, 2, 768), np.float32), 0.0, [B.Seg(700, page_table=t)])
    assert int(c.err.item()) == 1
    assert (m[..., 256:512] == 1).all() and (m[..., :256] != 1).any()
    c.err.zero_()


# ---------------------------------------------------------------- eviction
def evict64(c, keep, mass, pos, nxt, sink, recent):
    """New mass, positions and the pairs moved, by sorting."""
    mass, pos, moves = mass.copy(), pos.copy(), {}
    for s, L in enumerate(c.lengths):
        n = keep[s]
        for g in range(c.hkv):
            if n == L:
                moves[s, g] = np.zeros((0, 2), int)
                continue
            m, p = mass[s, g, :L].astype(np.float64), pos[s, g, :L]
            guard = (p < sink) | (p >= nxt[s] - recent)
            key = np.where(np.isnan(m), np.inf, m)
            tie = np.where(np.isnan(m), 1, 0)                # a NaN above infinity
            order = np.lexsort((np.arange(L), -tie, -key, ~guard))
            stays = np.zeros(L, bool)
            stays[order[:n]] = True
            dst = np.flatnonzero(~stays[:n])
            src = np.flatnonzero(stays[n:]) + n
            moves[s, g] = np.stack([src, dst], 1)
            mass[s, g, dst], pos[s, g, dst] = mass[s, g, src], pos[s, g, src]
            mass[s, g, n:L], pos[s, g, n:L] = 0, -1
    return mass, pos, moves


def move_rows(c, moves):
    for (s, g), mv in moves.items():
        for w in "kv":
            if c.cache.dtype == "fp4":
                got = fp4.get_rows(c.cache, c.segs[s], w, g, mv[:, 0])
                fp4.set_rows(c.cache, c.segs[s], w, g, mv[:, 1], *got)
            else:
                for a, b in mv:
                    arr, i = kvcache._store(c.cache, c.segs[s], w, g, int(a))
                    _, j = kvcache._store(c.cache, c.segs[s], w, g, int(b))
                    arr[j] = arr[i]


def same_cache(c):
    host = lambda t: (t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy())  # noqa: E731
    assert np.array_equal(host(c.k_pool), c.cache.k_pool) and np.array_equal(host(c.v_pool), c.cache.v_pool)
    for a, b in zip(c.gsegs, c.segs):
        if b.k_slab is not None:
            assert np.array_equal(host(a.k_slab), b.k_slab) and np.array_equal(host(a.v_slab), b.v_slab)


def check_evict(c, keep, mass, pos=None, nxt=None, sink=0, recent=0, cap=None):
    S, hkv = len(c.lengths), c.hkv
    cap = mass.shape[2]
    p0 = pos if pos is not None else np.broadcast_to(np.arange(cap, dtype=np.int32), mass.shape)
    n0 = nxt if nxt is not None else np.array(c.lengths)
    m2, p2, moves = evict64(c, keep, mass, p0, n0, sink, recent)
    dm, dp, mv = dev(mass), (dev(pos) if pos is not None else None), B.make_moves(S, hkv, cap)
    B.tfpa_evict_kv(c.gcache, c.gsegs, keep, dm, mv, key_pos=dp, next_pos=nxt, sink=sink, recent=recent)
    torch.cuda.synchronize()
    assert np.array_equal(dm.cpu().numpy().view(np.uint32), m2.view(np.uint32))
    if pos is not None:
        assert np.array_equal(dp.cpu().numpy(), p2)
    host = mv.cpu().numpy()
    for (s, g), want in moves.items():
        assert host[s, g, 0] == len(want)
        assert np.array_equal(host[s, g, 4: 4 + 2 * len(want)].reshape(-1, 2), want)
    move_rows(c, moves)
    same_cache(c)
    assert int(c.err.item()) == 0
    return m2, p2


def masses(c, seed=0, cap=None, zeros=0.1):
    rng = np.random.default_rng(seed)
    cap = cap or (max(c.lengths) + 7) // 4 * 4
    m = np.exp(2 * rng.standard_normal((len(c.lengths), c.hkv, cap))).astype(np.float32)
    m[rng.random(m.shape) < zeros] = 0
    return m


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("share", [0.02, 0.5, 0.97, 1.0])
def test_evict(kv, share):
    c = make(kv, [1300, 700, 257, 5], [True, False, True, False], seed=61)
    keep = np.array([max(1, int(L * share)) for L in c.lengths], np.int32)
    check_evict(c, keep, masses(c))


@pytest.mark.parametrize("L,n", [(2, 1), (3, 1), (3, 2), (1023, 512), (1024, 1023), (1025, 1), (2049, 1024), (2048, 2047), (5000, 2500)])
def test_evict_lengths(L, n):
    c = make("fp4", [L], [True], 2, 2, seed=62)
    check_evict(c, np.array([n], np.int32), masses(c, L))


@pytest.mark.parametrize("sink,recent", [(0, 1), (4, 0), (4, 64), (0, 300), (150, 150)])
def test_protected_positions(sink, recent):
    c = make("bf16", [700, 900], [True, False], seed=63)
    m = masses(c)
    m[:, :, :200] = 0                                        # what is protected would go first
    m2, p2 = check_evict(c, np.array([300, 400], np.int32), m, sink=sink, recent=recent)
    for s, (L, n) in enumerate(((700, 300), (900, 400))):
        kept = set(p2[s, 0, :n].tolist())
        assert set(range(sink)) <= kept and set(range(L - recent, L)) <= kept


def test_positions_of_their_own():
    """Positions with gaps and out of order, protected by position and not by slot."""
    c = make("fp8", [600, 333], [True, True], seed=64)
    rng = np.random.default_rng(1)
    cap = 604
    pos = np.full((2, 2, cap), -1, np.int32)
    for s, L in enumerate(c.lengths):
        for g in range(2):
            p = np.sort(rng.choice(5000, L, replace=False))
            pos[s, g, :L] = np.concatenate([rng.permutation(p[:-20]), p[-20:]])
    check_evict(c, np.array([200, 320], np.int32), masses(c, cap=cap), pos, np.array([5000, 5000], np.int32), sink=100, recent=90)


@pytest.mark.parametrize("kind", ["all_equal", "two_values", "nan_inf", "negative", "tiny"])
def test_ties_and_special_masses(kind):
    c = make("fp4", [1500], [True], 4, 4, seed=65)
    m = masses(c)
    rng = np.random.default_rng(4)
    if kind == "all_equal":
        m[:] = 3.25
    if kind == "two_values":
        m = np.where(rng.random(m.shape) < 0.3, np.float32(1), np.float32(0)) * np.where(rng.random(m.shape) < 0.5, -1, 1).astype(np.float32)
        m = np.abs(m) * np.where(m == 0, np.sign(rng.random(m.shape) - 0.5), 1).astype(np.float32)   # zeros of both signs
    if kind == "nan_inf":
        m[rng.random(m.shape) < 0.2] = np.nan
        m[rng.random(m.shape) < 0.2] = np.inf
    if kind == "negative":
        m -= 2
    if kind == "tiny":
        m *= np.float32(1e-42)
    check_evict(c, np.array([700], np.int32), m)


def test_evict_long_stream():
    c = make("fp8", [40001], [True], 1, 1, seed=66)
    check_evict(c, np.array([17777], np.int32), masses(c), sink=4, recent=100)


def test_evict_bad_page():
    c = make("bf16", [700], [True], 2, 1, seed=67)
    t = c.gsegs[0].page_table.clone()
    t[2] = -5
    m = np.zeros((1, 1, 700), np.float32)
    m[0, 0, 200:300] = np.arange(1, 101)                     # kept, moved within the good pages
    m[0, 0, 600:610] = 200                                   # kept, on the bad page
    before = c.k_pool.clone()
    B.tfpa_evict_kv(c.gcache, [B.Seg(700, page_table=t)], [110], dev(m), B.make_moves(1, 1, 700))
    torch.cuda.synchronize()
    assert int(c.err.item()) == 1
    bad = int(c.gsegs[0].page_table[2])
    assert torch.equal(before[bad], c.k_pool[bad])
    pt = c.gsegs[0].page_table.long()
    assert torch.equal(c.k_pool[pt[0], 0, 0], before[pt[0], 0, 200])
    c.err.zero_()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_serve_evict_and_go_on(kv):
    """A stream served, its weights summed, cut to half, and served on: the next tokens attend to exactly
    the kept keys; a second cut works on what the first left."""
    L, n, hq, hkv = 700, 350, 8, 2
    c = make(kv, [L], [True], hq, hkv, seed=68)
    table = c.gsegs[0].page_table
    seg_o = c.segs[0]
    cap = 1024
    mass, pos = torch.zeros(1, hkv, cap, device="cuda"), torch.full((1, hkv, cap), -1, dtype=torch.int32, device="cuda")
    pos[0, :, :L] = torch.arange(L, device="cuda", dtype=torch.int32)
    mv, sc = B.make_moves(1, hkv, cap), B.make_scratch(16, hq)
    rng = np.random.default_rng(7)

    def serve(length, rows, decay):
        rs, rp = np.zeros(rows, int), np.arange(length - rows, length)
        q = F.bf16_bits(rng.standard_normal((rows, hq, 128)))
        out, lse = torch.empty(rows, hq, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, hq, device="cuda")
        segs = [B.Seg(length, page_table=table)]
        B.tfpa_decode(c.gcache, segs, dev_bf16(q), rs, rp, SCALE, sc, out, lse)
        B.tfpa_key_mass(c.gcache, segs, dev_bf16(q), lse, rs, rp, SCALE, mass, decay=decay)
        return q, out, lse, rs, rp

    def store(at, count, next_pos):
        k, v = (F.bf16_bits(rng.standard_normal((count, hkv, 128))) for _ in range(2))
        segs = [B.Seg(at + count, page_table=table)]
        B.tfpa_write_kv(c.gcache, segs, dev_bf16(k), dev_bf16(v), np.zeros(count), np.arange(at, at + count))
        pos[0, :, at:at + count] = torch.arange(next_pos, next_pos + count, device="cuda", dtype=torch.int32)

    def check_row(length, served):
        q, out, lse, rs, rp = served
        host = lambda t: (t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy())  # noqa: E731
        c.cache.k_pool, c.cache.v_pool = host(c.k_pool), host(c.v_pool)
        seg_o.seq_len = length
        ref, rl, tol, lt = F.attend64(c.cache, [seg_o], q, rs, rp, SCALE)
        scale = 4 if kv == "bf16" else 1                     # P is rounded to bf16 there, 2^-8 of the weights
        F.assert_within(F.f64(out), ref, tol * scale + (2.0 ** -8 * np.abs(ref).max() if kv == "bf16" else 0), "served")

    check_row(L, serve(L, 6, 1.0))
    before = {(w, g): kvcache.gather(c.cache, seg_o, g, L)[w == "v"] for w in "kv" for g in range(hkv)}
    m0 = mass.cpu().numpy()[0].copy()
    B.tfpa_evict_kv(c.gcache, [B.Seg(L, page_table=table)], [n], mass, mv, key_pos=pos, sink=4, recent=32)
    kept = pos.cpu().numpy()[0, :, :n]
    for g in range(hkv):
        rest = np.setdiff1d(np.arange(4, L - 32), kept[g])
        chosen = np.intersect1d(np.arange(4, L - 32), kept[g])
        assert len(set(kept[g].tolist())) == n and m0[g][rest].max() <= m0[g][chosen].min()
        host = lambda t: (t.view(torch.int16).cpu().numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.cpu().numpy())  # noqa: E731
        c.cache.k_pool, c.cache.v_pool = host(c.k_pool), host(c.v_pool)
        seg_o.seq_len = n
        K, V = kvcache.gather(c.cache, seg_o, g, n)
        assert np.array_equal(K, before["k", g][kept[g]]) and np.array_equal(V, before["v", g][kept[g]])
    store(n, 40, L)
    check_row(n + 40, serve(n + 40, 3, 0.9))
    B.tfpa_evict_kv(c.gcache, [B.Seg(n + 40, page_table=table)], [200], mass, mv, key_pos=pos, next_pos=[L + 40], sink=4, recent=64)
    kept = pos.cpu().numpy()[0, :, :200]
    for g in range(hkv):
        # 24 of the 32 newest of the first round and the 40 new ones are the 64 newest
        assert set(range(4)) | set(range(L - 24, L + 40)) <= set(kept[g].tolist())
    store(200, 1, L + 40)
    check_row(201, serve(201, 1, 1.0))
    assert int(c.err.item()) == 0


def test_captured_and_replayed():
    """A step with its weights, and a cut, as CUDA graphs: the bytes of direct calls, call after call."""
    a, b = (make("fp4", [600, 500], [True, True], seed=69) for _ in range(2))
    q = dev_bf16(a.q(2))
    rs, rp = np.array([0, 1]), np.array([599, 499])
    runs = []
    for c in (a, b):
        mass, mv = torch.zeros(2, 2, 600, device="cuda"), B.make_moves(2, 2, 600)
        out, lse = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 8, device="cuda")
        sc = B.make_scratch(2, 8)

        def step(c=c, mass=mass, out=out, lse=lse, sc=sc):
            B.tfpa_decode(c.gcache, c.gsegs, q, rs, rp, SCALE, sc, out, lse)
            B.tfpa_key_mass(c.gcache, c.gsegs, q, lse, rs, rp, SCALE, mass, decay=0.5)

        def cut(c=c, mass=mass, mv=mv):
            B.tfpa_evict_kv(c.gcache, c.gsegs, [300, 499], mass, mv, sink=2, recent=10)
        runs.append((c, mass, mv, step, cut))
    c, mass, mv, step, cut = runs[0]
    s = torch.cuda.Stream()
    graphs = []
    for fn in (step, cut):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            fn()
        graphs.append(g)
    for _ in range(3):
        graphs[0].replay()
    graphs[1].replay()
    graphs[0].replay()
    torch.cuda.synchronize()
    _, mass2, mv2, step2, cut2 = runs[1]
    for _ in range(3):
        step2()
    cut2()
    step2()
    torch.cuda.synchronize()
    assert torch.equal(mass, mass2) and torch.equal(mv[..., 0], mv2[..., 0])
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)


# ---------------------------------------------------------------- many streams, long ones, other memory
def test_mass_of_many_slabs_and_pages():
    """More slab streams and more runs than a launch holds."""
    L = [40 + 7 * i for i in range(80)]
    c = make("fp4", L, [i % 3 == 0 for i in range(80)], 4, 2, seed=81)
    order = np.random.default_rng(1).permutation(80)
    check_mass(c, order, [L[s] - 1 for s in order], 0.5, "many")


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_mass_reads_pinned_host_rows(kv):
    c = make(kv, [500], [True], seed=82)
    q, lse = dev_bf16(c.q(3)), torch.randn(3, 8, device="cuda").abs() + 4
    m = [torch.zeros(1, 2, 512, device="cuda") for _ in range(2)]
    args = (np.zeros(3, int), np.arange(497, 500), SCALE)
    B.tfpa_key_mass(c.gcache, c.gsegs, q, lse, *args, m[0])
    B.tfpa_key_mass(c.gcache, c.gsegs, q.cpu().pin_memory(), lse.cpu().pin_memory(), *args, m[1])
    torch.cuda.synchronize()
    assert torch.equal(*m) and (m[0][..., :500] > 0).all()


def test_mass_of_rows_without_keys_and_bad_rows():
    """lse of -inf gives nothing; +inf gives nothing; a NaN reaches only its own heads' keys."""
    c = make("bf16", [300], [True], 8, 2, seed=83)
    q, lse = c.q(2), np.full((2, 8), 3.0, np.float32)
    lse[0, :4], lse[1, 1] = -np.inf, np.inf
    m = run_mass(c, q, lse, [0, 0], [298, 299], np.zeros((1, 2, 304), np.float32), 1.0)
    one = lse.copy()
    one[0, :], one[1, 1] = -np.inf, -np.inf
    want = run_mass(c, q, one, [0, 0], [298, 299], np.zeros((1, 2, 304), np.float32), 1.0)
    assert torch.equal(m[0, 0], want[0, 0]) and torch.isfinite(m).all()
    lse[0, 7] = np.nan
    m2 = run_mass(c, q, lse, [0, 0], [298, 299], np.zeros((1, 2, 304), np.float32), 1.0)
    assert torch.equal(m2[0, 0], m[0, 0]) and torch.isnan(m2[0, 1, :299]).all()
    assert (m2[0, :, 300:] == 0).all()


def test_evict_of_many_segments_and_heads():
    """More segments than a launch holds, and more kv heads than a cluster's CTAs."""
    L = [3 + 5 * i for i in range(140)]
    c = F.Fp4Case(L, [i % 2 == 0 for i in range(140)], 12, 12, seed=84).upload()
    check_evict(c, np.array([max(1, n * 2 // 3) for n in L], np.int32), masses(c, 3), sink=1)


@pytest.mark.parametrize("share", [0.1, 0.6])
def test_evict_of_a_stream_beyond_shared_memory(share):
    """More keys than a cluster holds: the choice reads the weights again."""
    L = 420001
    c = F.Fp4Case([L], [True], 1, 1, seed=85).upload()
    check_evict(c, np.array([int(L * share)], np.int32), masses(c, 4), recent=100)


def test_two_streams_evict_at_once():
    """Different caches on different streams: each its own answer."""
    cs = [F.Fp4Case([9000, 700], [True, False], 2, 2, seed=86 + i).upload() for i in range(2)]
    ms = [masses(c, i) for i, c in enumerate(cs)]
    keep = np.array([4000, 300], np.int32)
    dm = [dev(m) for m in ms]
    mv = [B.make_moves(2, 2, m.shape[2]) for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for c, m, w, s in zip(cs, dm, mv, streams):
        B.tfpa_evict_kv(c.gcache, c.gsegs, keep, m, w, stream=s)
    torch.cuda.synchronize()
    for c, m, d in zip(cs, ms, dm):
        p0 = np.broadcast_to(np.arange(m.shape[2], dtype=np.int32), m.shape)
        want, _, moves = evict64(c, keep, m, p0, np.array(c.lengths), 0, 0)
        assert np.array_equal(d.cpu().numpy(), want)
        move_rows(c, moves)
        same_cache(c)
