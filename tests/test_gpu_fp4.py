"""The 4-bit cache on the GPU: stored bytes against the oracle, attention against the formula in 64 bits,
and the invariants that the other cache types hold (paged or slab, batched or alone, sliced, appended,
planned: the same bytes)."""

import numpy as np
import pytest
import torch

from oracle import fp4, kvcache, kvstore
from paged_kv_cache_235_gb300 import binding as B
from paged_kv_cache_235_gb300 import workloads as wl
from tests.fp4_cases import SCALE, Fp4Case, assert_within, attend64, bf16_bits, dev, dev_bf16, f64

pytestmark = pytest.mark.gpu


def decode(c, q, rs, rp, cap=128, segs=None, fused=False, anc=None, max_splits=B.MAX_SPLITS):
    out = torch.full((len(rs), c.hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(rs), c.hq), float("nan"), device="cuda")
    sc = B.make_scratch(cap, c.hq, max_splits, fused_merge=fused)
    segs = segs or c.gsegs
    if anc is None:
        B.tfpa_decode(c.gcache, segs, dev_bf16(q), rs, rp, SCALE, sc, out, lse)
    else:
        a = dev(np.asarray(anc, np.uint64).view(np.int64))
        B.tfpa_decode_tree(c.gcache, segs, dev_bf16(q), rs, rp, a, SCALE, sc, out, lse)
    torch.cuda.synchronize()
    return out, lse


def check(c, q, rs, rp, out, lse, what="", anc=None):
    ref, rl, tol, ltol = attend64(c.cache, c.segs, q, rs, rp, SCALE, anc)
    assert_within(f64(out), ref, tol, what)
    assert_within(lse.cpu().numpy().astype(np.float64), rl, ltol, what + " lse")
    assert int(c.err.item()) == 0


def last_rows(lengths, R):
    return wl.decode_rows(lengths, R)


# ---------------------------------------------------------------- store and read
def _write_all(c):
    for s, L in enumerate(c.lengths):
        k = dev_bf16(c.k_bits[s].transpose(1, 0, 2))
        v = dev_bf16(c.v_bits[s].transpose(1, 0, 2))
        B.tfpa_write_kv(c.gcache, c.gsegs, k, v, np.full(L, s), np.arange(L))
    torch.cuda.synchronize()


@pytest.mark.parametrize("hq,hkv", [(8, 2), (5, 5), (4, 1)])
def test_stored_bytes_match_oracle(hq, hkv):
    c = Fp4Case([1, 255, 257, 700, 130], [True, True, False, True, False], hq, hkv, seed=11).upload()
    _write_all(c)
    c.fill().bytes_equal()
    assert int(c.err.item()) == 0


def test_special_values_are_stored_finite():
    def values(k, v):
        for x in (k[0], v[0]):
            x[0, 0, :8] = bf16_bits([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-38, -1e30, 3e38])
            x[0, 1, :] = bf16_bits(np.zeros(128))
            x[0, 2, :] = bf16_bits(np.full(128, np.nan))
            x[0, 3, 16:32] = bf16_bits(np.full(16, 1e-30))
    c = Fp4Case([40], [True], seed=12, values=values).upload()
    _write_all(c)
    c.fill().bytes_equal()
    k, v = torch.empty(40, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(40, 2, 128, dtype=torch.bfloat16, device="cuda")
    B.tfpa_read_kv(c.gcache, c.gsegs, k, v, np.zeros(40), np.arange(40))
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_rounding_ties_and_every_code():
    """Values on and next to every code border, under several scales."""
    def values(k, v):
        edge = np.array([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6, 0])
        for i in range(32):
            k[0][0, i] = bf16_bits(np.tile(edge, 8) * 2.0 ** (i - 16) * (-1) ** i)
            v[0][0, i] = bf16_bits(np.tile(np.roll(edge, i), 8) * (1 + i / 64))
    c = Fp4Case([64], [True], seed=13, values=values)
    c.cache.k_scale[:], c.cache.v_scale[:] = 1.0, 0.37
    c.upload()
    _write_all(c)
    c.fill().bytes_equal()


@pytest.mark.parametrize("device_pos", [True, False])
def test_rope_store_bytes_match_oracle(device_pos):
    c = Fp4Case([700, 300, 520], [True, False, True], seed=14).upload()
    cos, sin = wl.rope_table(1e6, 2048)
    rs, rp = np.array([0, 0, 1, 2, 2]), np.array([5, 699, 12, 300, 301])
    rpos = np.array([5, 3, 1000, 0, 2047], np.int32) if device_pos else rp
    k, v = bf16_bits(c.rng.standard_normal((5, 2, 128))), bf16_bits(c.rng.standard_normal((5, 2, 128)))
    B.tfpa_write_kv_rope(c.gcache, c.gsegs, dev_bf16(k), dev_bf16(v), rs, rp, dev(cos), dev(sin),
                         dev(rpos) if device_pos else None)
    for r in range(5):
        for g in range(2):
            kf = kvstore.rope_f32(k[r, g], cos[rpos[r]], sin[rpos[r]])
            for w, x, sc in (("k", kf, c.cache.k_scale), ("v", kvcache.bf16_to_f32(v[r, g]), c.cache.v_scale)):
                fp4.set_rows(c.cache, c.segs[rs[r]], w, g, np.array([rp[r]]), *(a[None] for a in fp4.quantise(x, sc[g])))
    c.bytes_equal()
    assert int(c.err.item()) == 0


def test_read_returns_the_stored_values():
    """Every row in a shuffled order; the product of exact code * block scale with the head's scale rounded
    to float32, then to bf16."""
    c = Fp4Case([300, 513], [True, False], 8, 4, seed=15).fill().upload()
    rs, rp = np.concatenate([np.zeros(300, int), np.ones(513, int)]), np.concatenate([np.arange(300), np.arange(513)])
    p = np.random.default_rng(1).permutation(813)
    rs, rp = rs[p], rp[p]
    out = [torch.empty(813, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.tfpa_read_kv(c.gcache, c.gsegs, *out, rs, rp)
    got = [o.view(torch.int16).cpu().numpy().view(np.uint16) for o in out]
    for g in range(4):
        for s, L in enumerate(c.lengths):
            at = rs == s
            for x, w, sc in ((got[0], "k", c.cache.k_scale), (got[1], "v", c.cache.v_scale)):
                codes, scales = fp4.get_rows(c.cache, c.segs[s], w, g, rp[at])
                want = (fp4.dequantise(codes, scales, 1.0).astype(np.float32) * sc[g]).astype(np.float32)
                assert np.array_equal(x[at, g], bf16_bits(want))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_read_of_the_other_cache_types(kv):
    from oracle import e4m3
    from tests.gpu_cases import GpuCase, fp8_scales
    from tests.oracle_cases import build_oracle_cache
    w = wl.small("batched_decode")
    w.kv_dtype = kv
    w.name += kv
    scales = fp8_scales(w) if kv == "fp8" else None
    g = GpuCase(w, scales)
    cache, segs = build_oracle_cache(w, *(scales or (None, None)))
    rs, rp = np.array([0, 1, 3, 3, 3]), np.array([0, 999, 255, 256, 511])
    k, v = (torch.empty(5, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.tfpa_read_kv(g.cache, g.segs, k, v, rs, rp)
    for r in range(5):
        for h in range(8):
            for t, which in ((k, "k"), (v, "v")):
                arr, idx = kvcache._store(cache, segs[rs[r]], which, h, rp[r])
                raw = arr[idx]
                if kv == "fp8":
                    sc = cache.k_scale if which == "k" else cache.v_scale
                    raw = bf16_bits((e4m3.decode(raw).astype(np.float32) * sc[h]).astype(np.float32))
                assert np.array_equal(t[r, h].view(torch.int16).cpu().numpy().view(np.uint16), raw)


def test_bad_page_is_flagged_and_its_rows_left():
    c = Fp4Case([700], [True], seed=16).fill().upload()
    t = c.gsegs[0].page_table.clone()
    t[1] = c.num_pages + 7
    seg = [B.Seg(700, page_table=t)]
    q = c.q(1)
    out, lse = decode(c, q, [0], [699], segs=seg)
    assert int(c.err.item()) == 1
    # the keys of the bad page take no part
    K = [kvcache.gather(c.cache, c.segs[0], g, 700) for g in range(2)]
    vis = np.r_[0:256, 512:700]
    for h in range(8):
        Kv, Vv = K[h // 4][0][vis], K[h // 4][1][vis]
        s = SCALE * Kv @ kvcache.bf16_to_f64(q[0, h])
        w = np.exp(s - s.max())
        assert np.abs(f64(out)[0, h] - w @ Vv / w.sum()).max() < 0.02
    c.err.zero_()
    k = torch.full((2, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    B.tfpa_read_kv(c.gcache, seg, k, k.clone(), [0, 0], [300, 5])
    assert int(c.err.item()) == 1 and (k[0] == 7).all() and not (k[1] == 7).all()


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (5, 1), (12, 2), (32, 8), (17, 1), (10, 2)])
@pytest.mark.parametrize("R", [1, 3])
def test_decode_group_sizes(hq, hkv, R):
    L = [700, 300, 1100]
    c = Fp4Case(L, [True, False, True], hq, hkv, seed=21).fill().upload()
    rs, rp = last_rows(L, R)
    q = c.q(len(rs))
    check(c, q, rs, rp, *decode(c, q, rs, rp), f"G={hq // hkv} R={R}")


@pytest.mark.parametrize("L", [1, 2, 17, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1024, 1025])
def test_lengths_around_tile_and_page_edges(L):
    c = Fp4Case([L, L], [True, False], seed=22).fill().upload()
    q = c.q(2)
    rs, rp = [0, 1], [L - 1, L - 1]
    out, lse = decode(c, q, rs, rp)
    check(c, q, rs, rp, out, lse, f"L={L}")
    fout, flse = decode(c, q, rs, rp, fused=True)
    assert torch.equal(out, fout) and torch.equal(lse, flse)


def test_long_stream_and_splits():
    L = [9001, 4097]
    c = Fp4Case(L, [True, True], 8, 2, seed=23).fill().upload()
    rs, rp = last_rows(L, 2)
    q = c.q(4)
    check(c, q, rs, rp, *decode(c, q, rs, rp), "long")


def test_rows_in_the_middle_and_out_of_order():
    """Rows that see few keys of their stream, twice the same row, positions going down."""
    c = Fp4Case([900, 600], [True, False], seed=24).fill().upload()
    rs, rp = np.array([0, 1, 0, 0, 0, 1]), np.array([899, 0, 300, 300, 5, 257])
    q = c.q(6)
    q[3] = q[2]
    out, lse = decode(c, q, rs, rp)
    check(c, q, rs, rp, out, lse, "middle")
    assert torch.equal(out[2], out[3])


@pytest.mark.parametrize("scale", [1e-4, 30.0])
def test_query_magnitudes(scale):
    """Flat weights, and weights on one key (a large running maximum)."""
    c = Fp4Case([777], [True], seed=25).fill().upload()
    q = c.q(2, scale)
    check(c, q, [0, 0], [775, 776], *decode(c, q, [0, 0], [775, 776]), f"q x {scale}")


def test_unwritten_rows_do_not_reach_the_output():
    """Rows behind the row's position hold anything: here the largest magnitudes and NaN scales."""
    c = Fp4Case([600], [True], seed=26).fill()
    for g in range(2):
        for w in ("k", "v"):
            fp4.set_rows(c.cache, c.segs[0], w, g, np.arange(301, 600), np.full((299, 64), 0x7F, np.uint8),
                         np.full((299, 8), 0x7E, np.uint8))
    c.upload()
    q = c.q(2)
    rs, rp = [0, 0], [299, 300]
    out, lse = decode(c, q, rs, rp)
    check(c, q, rs, rp, out, lse, "masked")
    short = [B.Seg(301, page_table=c.gsegs[0].page_table)]
    for g in range(2):                                      # and past the stream's end even NaN scales
        fp4.set_rows(c.cache, c.segs[0], "v", g, np.arange(301, 600), np.full((299, 64), 0x7F, np.uint8),
                     np.full((299, 8), 0x7F, np.uint8))
    c.v_pool.copy_(dev(c.cache.v_pool))
    out2, lse2 = decode(c, q, rs, rp, segs=short)
    check(c, q, rs, rp, out2, lse2, "NaN scales past the end")


def test_paged_slab_batched_and_sliced_give_the_same_bytes():
    L = [1300, 1300, 700]
    a = Fp4Case(L, [True, True, True], seed=27).fill().upload()
    b = Fp4Case(L, [False, False, True], seed=27).fill().upload()
    rs, rp = last_rows(L, 4)
    q = a.q(len(rs))
    out, lse = decode(a, q, rs, rp)
    o2, l2 = decode(b, q, rs, rp)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, l3 = decode(a, q, rs, rp, cap=3)
    assert torch.equal(out, o3) and torch.equal(lse, l3)
    for s in range(3):
        at = np.flatnonzero(rs == s)
        o4, l4 = decode(a, q[at], rs[at], rp[at])
        assert torch.equal(out[torch.from_numpy(at).cuda()], o4)


@pytest.mark.parametrize("nodes", [2, 7, 20, 64])
def test_tree(nodes):
    L = [700, 65]
    c = Fp4Case(L, [True, False], seed=28).fill().upload()
    rs, rp = last_rows(L, min(nodes, 64))
    anc = [m for s in range(2) for m in wl.tree_masks(wl.random_tree(nodes, 5 + s))]
    q = c.q(len(rs))
    check(c, q, rs, rp, *decode(c, q, rs, rp, anc=anc), f"tree {nodes}", anc)
    full = [wl.ALL_VISIBLE] * len(rs)
    out, _ = decode(c, q, rs, rp, anc=full)
    ref, _ = decode(c, q, rs, rp)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("R", [12, 13, 40, 130])
def test_many_rows_of_a_stream(R):
    c = Fp4Case([500], [True], 8, 2, seed=29).fill().upload()
    rs, rp = last_rows([500], R)
    q = c.q(R)
    check(c, q, rs, rp, *decode(c, q, rs, rp), f"R={R}")
    # the two halves of the call, with each row's split count
    sc = B.make_scratch(R, 8, fused_merge=False)
    B.tfpa_decode_partial(c.gcache, c.gsegs, dev_bf16(q), rs, rp, SCALE, sc)
    out = torch.empty(R, 8, 128, dtype=torch.bfloat16, device="cuda")
    B.tfpa_merge(sc, 8, B.tfpa_row_splits(c.gcache, c.gsegs, rs, rp), out)
    assert torch.equal(out, decode(c, q, rs, rp)[0])


@pytest.mark.parametrize("R,fused", [(1, False), (1, True), (3, True), (14, False)])
def test_append_is_write_then_decode(R, fused):
    L = [1000, 257, 130]
    a = Fp4Case(L, [True, False, True], seed=30).fill().upload()
    b = Fp4Case(L, [True, False, True], seed=30).fill().upload()
    rs, rp = last_rows(L, R)
    k, v = (dev_bf16(bf16_bits(a.rng.standard_normal((len(rs), 2, 128)))) for _ in range(2))
    q = a.q(len(rs))
    B.tfpa_write_kv(b.gcache, b.gsegs, k, v, rs, rp)
    ref, rlse = decode(b, q, rs, rp, fused=fused)
    out, lse = torch.empty_like(ref), torch.empty_like(rlse)
    sc = B.make_scratch(128, 8, fused_merge=fused)
    B.tfpa_decode_append(a.gcache, a.gsegs, k, v, dev_bf16(q), rs, rp, SCALE, sc, out, lse)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rlse)
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)
    assert torch.equal(a.gsegs[1].k_slab, b.gsegs[1].k_slab) and torch.equal(a.gsegs[1].v_slab, b.gsegs[1].v_slab)


def test_static_scratch():
    c = Fp4Case([900], [True], seed=31).fill().upload()
    q = c.q(2)
    ref, rl = decode(c, q, [0, 0], [898, 899])
    out, lse = torch.empty_like(ref), torch.empty_like(rl)
    B.tfpa_decode_static(c.gcache, c.gsegs, dev_bf16(q), [0, 0], [898, 899], SCALE, out, lse)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_planned_loop_replayed_as_a_graph():
    """Five steps, lengths growing past a page, on one captured graph: the bytes of direct calls."""
    cap, L0 = 520, 253
    a = Fp4Case([cap, cap], [True, False], seed=32).fill().upload()
    b = Fp4Case([cap, cap], [True, False], seed=32).fill().upload()
    rng = np.random.default_rng(3)
    k, v = (torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    sc, sc2 = B.make_scratch(8, 8), B.make_scratch(8, 8)
    tab = B.SegTable([B.Seg(L0, page_table=a.gsegs[0].page_table),
                      B.Seg(L0, k_slab=a.gsegs[1].k_slab, v_slab=a.gsegs[1].v_slab, slab_cap=768)])
    host = torch.zeros(1 << 15, dtype=torch.uint8).pin_memory()
    dyn = torch.zeros(1 << 15, dtype=torch.uint8, device="cuda")
    plan = B.Plan()
    plan.set_device(dyn)
    s = torch.cuda.Stream()
    rs = np.array([0, 1])
    for step in range(5):
        n = L0 + 1 + step
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape))).to(torch.bfloat16))
        for i in range(2):
            tab.set_seq_len(i, n)
        plan.clear()
        plan.decode_append(a.gcache, tab, k, v, q, rs, np.array([n - 1, n - 1]), SCALE, sc, out)
        plan.pack(host)
        torch.cuda.synchronize()
        if step == 0:
            dyn.copy_(host)
            plan.launch()
            torch.cuda.synchronize()
            plan.capture(before=[(dyn, host, plan.dyn_bytes())], stream=s)
        plan.replay(s)
        s.synchronize()
        segs = [B.Seg(n, page_table=b.gsegs[0].page_table),
                B.Seg(n, k_slab=b.gsegs[1].k_slab, v_slab=b.gsegs[1].v_slab, slab_cap=768)]
        ref = torch.empty_like(out)
        B.tfpa_decode_append(b.gcache, segs, k, v, q, rs, [n - 1, n - 1], SCALE, sc2, ref)
        torch.cuda.synchronize()
        assert torch.equal(out, ref), step
    assert torch.equal(a.k_pool, b.k_pool)


# ---------------------------------------------------------------- upkeep
def test_keep_moves_codes_and_scales():
    c = Fp4Case([700, 300, 520], [True, False, True], seed=33).fill().upload()
    ks, src, dst = [0, 0, 1, 1, 2], [10, 3, 7, 8, 100], [3, 11, 8, 7, 400]
    B.tfpa_keep_kv(c.gcache, c.gsegs, ks, src, dst)
    got = {(i, w, g): fp4.get_rows(c.cache, c.segs[s], w, g, np.array([p]))
           for i, (s, p) in enumerate(zip(ks, src)) for w in "kv" for g in range(2)}
    for i, (s, p) in enumerate(zip(ks, dst)):
        for w in "kv":
            for g in range(2):
                fp4.set_rows(c.cache, c.segs[s], w, g, np.array([p]), *got[i, w, g])
    c.bytes_equal()


@pytest.mark.parametrize("pinned", [False, True])
@pytest.mark.parametrize("p0,p1", [(0, 700), (5, 6), (127, 130), (250, 515)])
def test_save_and_restore(p0, p1, pinned):
    c = Fp4Case([700, 300], [True, False], seed=34).fill().upload()
    n = p1 - p0
    for s in range(2):
        if p1 > c.lengths[s]:
            continue
        img = torch.zeros(2 * 2 * n * 72, dtype=torch.uint8)
        img = img.pin_memory() if pinned else img.cuda()
        B.tfpa_save_kv(c.gcache, c.gsegs[s], p0, p1, img)
        torch.cuda.synchronize()
        host = img.cpu().numpy()
        codes, scales = host[: 4 * n * 64].reshape(2, 2, n, 64), host[4 * n * 64:].reshape(2, 2, n, 8)
        for wi, w in enumerate("kv"):
            for g in range(2):
                a, b = fp4.get_rows(c.cache, c.segs[s], w, g, np.arange(p0, p1))
                assert np.array_equal(codes[wi, g], a) and np.array_equal(scales[wi, g], b)
        before = [t.clone() for t in (c.k_pool, c.v_pool)]
        zero = torch.zeros(n, 2, 128, dtype=torch.bfloat16, device="cuda")
        B.tfpa_write_kv(c.gcache, c.gsegs, zero, zero, np.full(n, s), np.arange(p0, p1))
        B.tfpa_restore_kv(c.gcache, c.gsegs[s], p0, p1, img)
        assert torch.equal(c.k_pool, before[0]) and torch.equal(c.v_pool, before[1])
        c.bytes_equal()


def test_offsets_past_32_bits():
    """A pool of more than 2^31 bytes: rows in its last pages are stored, read and attended."""
    hkv, num = 8, 16384                                     # 2.4 GB each for K and V
    kp, vp = (torch.zeros(num, hkv, fp4.BLOCK, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Fp4Case([600], [True], 8, 8, seed=35)
    pages = np.array([num - 1, 3, num - 2], np.int32)
    cache = B.Cache("fp4", 8, hkv, kp, vp, dev(c.cache.k_scale), dev(c.cache.v_scale), None, num)
    seg = [B.Seg(600, page_table=dev(pages))]
    k, v = dev_bf16(c.k_bits[0].transpose(1, 0, 2)), dev_bf16(c.v_bits[0].transpose(1, 0, 2))
    B.tfpa_write_kv(cache, seg, k, v, np.zeros(600), np.arange(600))
    q = c.q(1)
    out = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda")
    B.tfpa_decode(cache, seg, dev_bf16(q), [0], [599], SCALE, B.make_scratch(1, 8), out)
    ref, _, tol, _ = attend64(c.fill().cache, c.segs, q, [0], [599], SCALE)
    assert_within(f64(out), ref, tol, "far pages")
    assert bool((kp[num - 1] != 0).any()) and not bool((kp[num - 3] != 0).any())


# ---------------------------------------------------------------- prompt chunks
def prefill(c, q, rs, rp, max_rows=0, segs=None):
    out = torch.full((len(rs), c.hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((len(rs), c.hq), float("nan"), device="cuda")
    B.tfpa_prefill(c.gcache, segs or c.gsegs, dev_bf16(q), rs, rp, SCALE, out, lse, max_rows_per_launch=max_rows)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (5, 1)])
@pytest.mark.parametrize("prefix,chunk", [(0, 1), (0, 128), (0, 129), (300, 257), (1000, 70), (127, 130), (513, 1)])
def test_prompt_chunks(hq, hkv, prefix, chunk):
    L = prefix + chunk
    c = Fp4Case([L, L], [True, False], hq, hkv, seed=41).fill().upload()
    rs, rp = last_rows([L, L], chunk)
    q = c.q(len(rs))
    out, lse = prefill(c, q, rs, rp)
    check(c, q, rs, rp, out, lse, f"chunk {prefix}+{chunk}")
    o2, l2 = prefill(c, q, rs, rp, max_rows=128)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_prompt_chunk_ignores_unwritten_rows():
    c = Fp4Case([500], [True], seed=42).fill()
    for g in range(2):
        for w in ("k", "v"):
            fp4.set_rows(c.cache, c.segs[0], w, g, np.arange(333, 500), np.full((167, 64), 0x7F, np.uint8),
                         np.full((167, 8), 0x7F, np.uint8))
    c.upload()
    seg = [B.Seg(333, page_table=c.gsegs[0].page_table)]
    q = c.q(200)
    rs, rp = np.zeros(200, np.int32), np.arange(133, 333)
    out, lse = prefill(c, q, rs, rp, segs=seg)
    check(c, q, rs, rp, out, lse, "unwritten")


def test_prompt_chunk_with_a_bad_page():
    c = Fp4Case([700], [True], seed=43).fill().upload()
    t = c.gsegs[0].page_table.clone()
    t[1] = -1
    q = c.q(130)
    rs, rp = np.zeros(130, np.int32), np.arange(570, 700)
    out, lse = prefill(c, q, rs, rp, segs=[B.Seg(700, page_table=t)])
    assert int(c.err.item()) == 1 and torch.isfinite(out.float()).all()
    c.err.zero_()
    ref, _ = decode(c, q, rs, rp, segs=[B.Seg(700, page_table=t)], cap=130)
    assert (out.float() - ref.float()).abs().max() < 0.05
    c.err.zero_()


def test_a_stream_served_in_four_bits():
    """A prompt stored with its rotary positions in two chunks, each attended, then four tokens appended:
    every output against the formula on the bytes the cache holds."""
    from paged_kv_cache_235_gb300 import workloads as wl
    c = Fp4Case([704], [True], seed=44).upload()
    cos, sin = wl.rope_table(1e4, 1024)
    cos, sin = dev(cos), dev(sin)
    k, v = dev_bf16(c.k_bits[0].transpose(1, 0, 2)), dev_bf16(c.v_bits[0].transpose(1, 0, 2))
    q = c.q(704)
    t = c.gsegs[0].page_table
    got = []
    for a, b in ((0, 300), (300, 700)):
        at = np.arange(a, b)
        B.tfpa_write_kv_rope(c.gcache, [B.Seg(b, page_table=t)], k[a:b], v[a:b], np.zeros(b - a), at, cos, sin)
        got.append(prefill(c, q[a:b], np.zeros(b - a), at, segs=[B.Seg(b, page_table=t)]))
    sc = B.make_scratch(4, 8)
    for p in range(700, 704):
        out, lse = torch.empty(1, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 8, device="cuda")
        B.tfpa_decode_append(c.gcache, [B.Seg(p + 1, page_table=t)], k[p:p + 1], v[p:p + 1], dev_bf16(q[p:p + 1]), [0], [p],
                             SCALE, sc, out, lse)
        got.append((out, lse))
    torch.cuda.synchronize()
    c.cache.k_pool, c.cache.v_pool = c.k_pool.cpu().numpy(), c.v_pool.cpu().numpy()
    out, lse = torch.cat([o for o, _ in got]), torch.cat([x for _, x in got])
    check(c, q, np.zeros(704, int), np.arange(704), out, lse, "served")


# ---------------------------------------------------------------- calls that mix and overlap
@pytest.mark.parametrize("hq,hkv", [(32, 8), (8, 2), (5, 1), (8, 1)])
def test_one_call_of_short_and_long_runs(hq, hkv):
    """Runs for all three kernels in one call: the bytes of each run alone, and the formula."""
    L, R = [900, 1300, 4500, 700, 333], [1, 2, 30, 4, 9]
    c = Fp4Case(L, [True, False, True, True, False], hq, hkv, seed=71).fill().upload()
    rs = np.concatenate([np.full(r, s) for s, r in enumerate(R)])
    rp = np.concatenate([np.arange(n - r, n) for n, r in zip(L, R)])
    q = c.q(len(rs))
    out, lse = decode(c, q, rs, rp)
    check(c, q, rs, rp, out, lse, f"{hq}/{hkv}")
    for s in range(len(L)):
        at = np.flatnonzero(rs == s)
        o1, l1 = decode(c, q[at], rs[at], rp[at])
        assert torch.equal(o1, out[at[0]: at[-1] + 1]) and torch.equal(l1, lse[at[0]: at[-1] + 1])


def test_halves_of_a_mixed_call():
    """tfpa_decode_partial and tfpa_merge with each row's own split count: the bytes of tfpa_decode."""
    L, R = [9000, 2500, 4000], [1, 5, 20]
    c = Fp4Case(L, [True, True, False], 16, 4, seed=72).fill().upload()
    rs = np.concatenate([np.full(r, s) for s, r in enumerate(R)])
    rp = np.concatenate([np.arange(n - r, n) for n, r in zip(L, R)])
    q = c.q(len(rs))
    out, lse = decode(c, q, rs, rp)
    check(c, q, rs, rp, out, lse)
    sc = B.make_scratch(64, 16, fused_merge=False)
    ns = B.tfpa_row_splits(c.gcache, c.gsegs, rs, rp)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    B.tfpa_decode_partial(c.gcache, c.gsegs, dev_bf16(q), rs, rp, SCALE, sc)
    B.tfpa_merge(sc, 16, ns, o2, l2)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_long_run_with_a_bad_page():
    """Verify rows: the keys of a page outside the pool take no part, on either kind of tile."""
    c = Fp4Case([1500], [True], 8, 2, seed=73).fill().upload()
    t = c.gsegs[0].page_table.clone()
    t[2] = -7
    rs, rp = np.zeros(20, int), np.arange(1480, 1500)
    q = c.q(20)
    out, lse = decode(c, q, rs, rp, segs=[B.Seg(1500, page_table=t)])
    assert int(c.err.item()) == 1
    c.err.zero_()
    qd, keep = f64(dev_bf16(q)), np.r_[0:512, 768:1500]
    for g in range(2):
        K, V = kvcache.gather(c.cache, c.segs[0], g, 1500)
        for r in range(20):
            vis = keep[keep <= rp[r]]
            for h in range(4 * g, 4 * g + 4):
                x = SCALE * (K[vis] @ qd[r, h])
                w = np.exp(x - x.max())
                ref = w @ V[vis] / w.sum()
                tol = 2.0 ** -9 * (w @ np.abs(V[vis]) / w.sum()) + 2.0 ** -8 * np.abs(ref) + 1e-6
                assert (np.abs(f64(out[r, h]) - ref) <= tol).all()


def test_another_stream_and_two_threads():
    """Calls on streams of their own from two threads at once: the bytes of the same calls one by one."""
    import threading
    jobs = []
    for i in range(2):
        c = Fp4Case([3000 + 100 * i, 800], [True, False], 8, 2, seed=74 + i).fill().upload()
        rs = np.concatenate([np.zeros(1 + 19 * i, int), np.ones(2, int)])
        rp = np.concatenate([np.arange(c.lengths[0] - 1 - 19 * i, c.lengths[0]), [798, 799]])
        q = c.q(len(rs))
        jobs.append((c, rs, rp, dev_bf16(q), decode(c, q, rs, rp)))
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            c, rs, rp, q, _ = jobs[i]
            stream = torch.cuda.Stream()
            out = torch.full((len(rs), 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
            lse = torch.full((len(rs), 8), float("nan"), device="cuda")
            sc = B.make_scratch(64, 8)
            torch.cuda.synchronize()
            for _ in range(20):
                B.tfpa_decode(c.gcache, c.gsegs, q, rs, rp, SCALE, sc, out, lse, stream=stream)
            stream.synchronize()
            got[i] = (out, lse)
        except Exception as e:                                # shown by the assertion below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for i in range(2):
        assert torch.equal(got[i][0], jobs[i][4][0]) and torch.equal(got[i][1], jobs[i][4][1])


def test_pinned_host_rows():
    """Read-back into pinned host memory; decode's q there (short runs), refused for verify tiles."""
    c = Fp4Case([600], [True], 8, 2, seed=76).fill().upload()
    rp = np.array([599, 0, 256])
    k, v = (torch.empty(3, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kh, vh = (torch.empty(3, 2, 128, dtype=torch.bfloat16).pin_memory() for _ in range(2))
    B.tfpa_read_kv(c.gcache, c.gsegs, k, v, np.zeros(3), rp)
    B.tfpa_read_kv(c.gcache, c.gsegs, kh, vh, np.zeros(3), rp)
    torch.cuda.synchronize()
    assert torch.equal(k.cpu(), kh) and torch.equal(v.cpu(), vh)
    q = c.q(5)
    out, lse = decode(c, q, np.zeros(5, int), np.arange(595, 600))
    qh = dev_bf16(q).cpu().pin_memory()
    o2, sc = torch.empty_like(out), B.make_scratch(16, 8)
    with pytest.raises(B.TfpaError):
        B.tfpa_decode(c.gcache, c.gsegs, qh, np.zeros(5, int), np.arange(595, 600), SCALE, sc, o2)
    o1, _ = decode(c, q[:4], np.zeros(4, int), np.arange(595, 599))
    B.tfpa_decode(c.gcache, c.gsegs, qh[:4], np.zeros(4, int), np.arange(595, 599), SCALE, sc, o2[:4])
    torch.cuda.synchronize()
    assert torch.equal(o1, o2[:4])
