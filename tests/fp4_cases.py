"""Set-up of 4-bit caches for the tests: the oracle's bytes, uploaded as they are, and a plain
attention in 64 bits with the bound that the kernels' roundings allow."""

import numpy as np
import torch

from oracle import fp4, kvcache
from paged_kv_cache_235_gb300 import binding as B
from paged_kv_cache_235_gb300 import workloads as wl

SCALE = 1 / 128 ** 0.5


def bf16_bits(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(dtype) if dtype is not None else t).cuda()


def dev_bf16(bits):
    return dev(np.ascontiguousarray(bits).view(np.int16), torch.bfloat16)


class Fp4Case:
    """Streams of a 4-bit cache on the host (oracle) and, on demand, the GPU.  Everything that no
    stream's row covers holds random bytes, NaN scales among them."""

    def __init__(self, lengths, paged, hq=8, hkv=2, seed=1, slack=2, values=None):
        self.lengths, self.hq, self.hkv = list(lengths), hq, hkv
        rng = np.random.default_rng(seed)
        pages = [(L + 255) // 256 for L in lengths]
        self.num_pages = sum(n for n, p in zip(pages, paged) if p) + slack
        tables = wl.permuted_tables(list(lengths), list(paged), self.num_pages, seed)
        k, v = [], []
        for L in lengths:
            k.append(bf16_bits(rng.standard_normal((hkv, L, 128)) * (1 + 3 * (rng.random(128) < 0.1))))
            v.append(bf16_bits(rng.standard_normal((hkv, L, 128)) * (1 + 3 * (rng.random(128) < 0.1))))
        if values is not None:
            values(k, v)
        self.k_bits, self.v_bits = k, v
        f = kvcache.bf16_to_f32
        amax = lambda xs: np.nanmax([np.nanmax(np.where(np.isfinite(f(x)), np.abs(f(x)), 0), axis=(1, 2)) for x in xs], axis=0)  # noqa: E731
        ks, vs = (amax(k) / 2688).astype(np.float32), (amax(v) / 2688).astype(np.float32)
        junk = lambda *s: rng.integers(0, 256, s, dtype=np.uint8)  # noqa: E731
        self.cache = kvcache.Cache("fp4", hkv, 128, junk(self.num_pages, hkv, fp4.BLOCK),
                                   junk(self.num_pages, hkv, fp4.BLOCK), ks, vs)
        self.segs = []
        for L, n, p, t in zip(lengths, pages, paged, tables):
            if p:
                self.segs.append(kvcache.Segment(L, page_table=t))
            else:
                self.segs.append(kvcache.Segment(L, k_slab=junk(hkv, n, fp4.BLOCK), v_slab=junk(hkv, n, fp4.BLOCK)))
        self.rng = rng

    def fill(self):
        for s, seg in enumerate(self.segs):
            for g in range(self.hkv):
                for w, x, sc in (("k", self.k_bits[s], self.cache.k_scale), ("v", self.v_bits[s], self.cache.v_scale)):
                    codes, scales = fp4.quantise(kvcache.bf16_to_f32(x[g]), sc[g])
                    fp4.set_rows(self.cache, seg, w, g, np.arange(seg.seq_len), codes, scales)
        return self

    def upload(self):
        c = self.cache
        self.k_pool, self.v_pool = dev(c.k_pool), dev(c.v_pool)
        self.k_scale, self.v_scale = dev(c.k_scale), dev(c.v_scale)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.gcache = B.Cache("fp4", self.hq, self.hkv, self.k_pool, self.v_pool, self.k_scale, self.v_scale,
                              self.err, self.num_pages)
        self.gsegs = []
        for seg in self.segs:
            if seg.page_table is not None:
                self.gsegs.append(B.Seg(seg.seq_len, page_table=dev(seg.page_table),
                                        page_table_host=np.asarray(seg.page_table, np.int32)))
            else:
                self.gsegs.append(B.Seg(seg.seq_len, k_slab=dev(seg.k_slab), v_slab=dev(seg.v_slab),
                                        slab_cap=seg.k_slab.shape[1] * 256))
        return self

    def bytes_equal(self):
        """The GPU's cache holds the oracle's bytes, everywhere."""
        assert np.array_equal(self.k_pool.cpu().numpy(), self.cache.k_pool)
        assert np.array_equal(self.v_pool.cpu().numpy(), self.cache.v_pool)
        for gs, os_ in zip(self.gsegs, self.segs):
            if os_.k_slab is not None:
                assert np.array_equal(gs.k_slab.cpu().numpy(), os_.k_slab)
                assert np.array_equal(gs.v_slab.cpu().numpy(), os_.v_slab)

    def q(self, rows, scale=1.0):
        return bf16_bits(self.rng.standard_normal((rows, self.hq, 128)) * scale)


def attend64(cache, segs, q_bits, row_seg, row_pos, scale, row_anc=None):
    """out, lse and the allowance of each output element for the kernels' roundings, in 64 bits.

    A weight is off by its f16 (or bf16) rounding, 2^-11 (the operands' products are exact), and by what
    a float32 sum of 128 products allows its score, 128 2^-24 sum |q k| scale, plus 2^-20 for the
    exponential; below 2^-14 a weight rounds to a multiple of 2^-24 against a largest weight of at least
    1.  All of it weighs |v|; the output then rounds to bf16, 2^-8."""
    rows, hq, d = q_bits.shape
    G = hq // cache.hkv
    q = kvcache.bf16_to_f64(q_bits)
    out, lse, tol = np.zeros((rows, hq, d)), np.zeros((rows, hq)), np.zeros((rows, hq, d))
    ltol = np.zeros((rows, hq))
    for s in sorted(set(int(x) for x in row_seg)):
        rs = [r for r in range(rows) if row_seg[r] == s]
        n = max(int(row_pos[r]) for r in rs) + 1
        for g in range(cache.hkv):
            K, V = kvcache.gather(cache, segs[s], g, n)
            for r in rs:
                p = int(row_pos[r])
                vis = np.arange(n) <= p
                if row_anc is not None:
                    back = p - np.arange(n)
                    bit = (int(row_anc[r]) >> np.clip(back, 0, 63).astype(object)) & 1
                    vis &= (back > 63) | (bit.astype(np.int64) == 1)
                Kv, Vv = K[vis], V[vis]
                Q = q[r, g * G:(g + 1) * G]
                S = scale * (Q @ Kv.T)
                Sabs = scale * (np.abs(Q) @ np.abs(Kv).T)
                m = S.max(1, keepdims=True)
                E = np.exp(S - m)
                Z = E.sum(1, keepdims=True)
                W = E / Z
                es = 2 * 128 * 2.0 ** -24 * Sabs.max(1, keepdims=True) + 2.0 ** -20
                h = slice(g * G, (g + 1) * G)
                out[r, h] = W @ Vv
                lse[r, h] = m[:, 0] + np.log(Z[:, 0])
                A = W @ np.abs(Vv)
                tol[r, h] = (2.0 ** -8 * np.abs(out[r, h]) + A * (2.0 ** -11 + 2 * es)
                             + len(Vv) * 2.0 ** -25 / Z * np.abs(Vv).max() + 1e-30)
                ltol[r, h] = es[:, 0] + 2.0 ** -22 * (np.abs(lse[r, h]) + np.abs(m[:, 0]) + 20)
    return out, lse, tol, ltol


def assert_within(got, ref, tol, what=""):
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what + ": not finite"
    if not (err <= tol).all():
        i = np.unravel_index(np.argmax(err / tol), err.shape)
        raise AssertionError(f"{what}: {(err > tol).sum()} of {err.size} outside; worst at {i}: got {got[i]} "
                             f"ref {ref[i]} allowed {tol[i]}")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)
