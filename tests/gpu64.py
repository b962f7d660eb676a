"""Long caches for the GPU tests, filled on the GPU with random stored bytes, and attention and attention weight
over them in 64 bits on the GPU, with the allowances that the kernels' roundings need (those of fp4_cases.attend64
and of test_gpu_evict.mass64)."""

import numpy as np
import torch

from paged_kv_cache_235_gb300 import binding as B

SCALE = 1 / 128 ** 0.5
U = 2.0 ** -24                                   # half a float32 step


class LongCase:
    """Streams of stored bytes: finite in every row that a stream has, anything behind its end."""

    def __init__(self, kv, lengths, paged, hq, hkv, seed):
        self.kv, self.lengths, self.hq, self.hkv = kv, list(lengths), hq, hkv
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g = g
        pages = [-(-L // 256) for L in lengths]
        total = sum(n for n, p in zip(pages, paged) if p)
        self.num_pages = total + 3
        perm = torch.randperm(self.num_pages, generator=g, device="cuda").to(torch.int32)
        self.k_pool, self.v_pool = (self._bytes(self.num_pages, hkv) for _ in range(2))
        self.k_scale = 0.2 + 0.2 * torch.rand(hkv, generator=g, device="cuda")
        self.v_scale = 0.2 + 0.2 * torch.rand(hkv, generator=g, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        sc = (None, None) if kv == "bf16" else (self.k_scale, self.v_scale)
        self.cache = B.Cache(kv, hq, hkv, self.k_pool, self.v_pool, *sc, self.err, self.num_pages)
        self.segs, self.slabs, at = [], {}, 0
        for s, (L, n, p) in enumerate(zip(lengths, pages, paged)):
            if p:
                self.segs.append(B.Seg(L, page_table=perm[at:at + n].contiguous()))
                at += n
            else:
                k, v = (self._bytes(n, hkv).transpose(0, 1).contiguous() for _ in range(2))
                self.slabs[s] = (k, v)
                self.segs.append(B.Seg(L, k_slab=k, v_slab=v, slab_cap=256 * n))
        for s, L in enumerate(lengths):          # what lies behind a stream's end
            if L % 256:
                for w in (0, 1):
                    self._spoil(s, w, pages[s] - 1, L % 256)

    def _bytes(self, pages, hkv):
        r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=self.g, device="cuda", dtype=torch.uint8)  # noqa: E731
        if self.kv == "bf16":
            return torch.randn(pages, hkv, 256, 128, generator=self.g, device="cuda").to(torch.bfloat16)
        if self.kv == "fp8":                     # magnitudes up to 15
            return r(0, 0x58, pages, hkv, 256, 128) | (r(0, 2, pages, hkv, 256, 128) << 7)
        x = r(0, 256, pages, hkv, 2, 9216)
        x[..., 8192:] = r(0x28, 0x40, pages, hkv, 2, 1024)       # scales of 0.25 to 1.9
        return x.reshape(pages, hkv, B.FP4_BLOCK)

    def _page(self, s, w, page):
        """Stored bytes of one page of every kv head, as a view."""
        if s in self.slabs:
            return self.slabs[s][w][:, page]
        return (self.v_pool if w else self.k_pool)[int(self.segs[s].page_table[page])]

    def _spoil(self, s, w, page, first):
        blk = self._page(s, w, page)
        if self.kv == "bf16":
            blk[:, first:] = float("nan")
        elif self.kv == "fp8":
            blk[:, first:] = 0x7F
        else:
            h = blk.view(self.hkv, 2, 9216)
            sc = h[..., 8192:].unflatten(-1, (128, 8))
            for half in (0, 1):
                sc[:, half, max(0, first - 128 * half):] = 0x7F

    def values(self, s, w, g):
        """K (w = 0) or V of stream s, kv head g: float64 [L][128]."""
        if s in self.slabs:
            x = self.slabs[s][w][g]
        else:
            x = (self.v_pool if w else self.k_pool)[self.segs[s].page_table.long(), g]
        L = self.lengths[s]
        if self.kv == "bf16":
            return x.reshape(-1, 128)[:L].double()
        sc = (self.v_scale if w else self.k_scale)[g].double()
        if self.kv == "fp8":
            return x.reshape(-1, 128)[:L].contiguous().view(torch.float8_e4m3fn).double() * sc
        h = x.reshape(-1, 9216)
        code, scale = h[:, :8192].reshape(-1, 64)[:L].long(), h[:, 8192:].reshape(-1, 8)[:L]
        mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
        lut = torch.cat([mag, -mag])
        v = torch.stack([lut[code % 16], lut[code // 16]], -1).reshape(L, 8, 16)
        return (v * scale.contiguous().view(torch.float8_e4m3fn).double()[..., None]).reshape(L, 128) * sc

    def q(self, rows, scale=1.0):
        return (torch.randn(rows, self.hq, 128, generator=self.g, device="cuda") * scale).to(torch.bfloat16)


def last_rows(lengths, counts):
    """Row tables of each stream's last counts[s] positions."""
    rs = np.repeat(np.arange(len(lengths), dtype=np.int32), counts)
    rp = np.concatenate([np.arange(L - n, L, dtype=np.int32) for L, n in zip(lengths, counts)])
    return rs, rp


def _rows(c, rs, rp, anc):
    for s in sorted(set(int(x) for x in rs)):
        at = np.flatnonzero(rs == s)
        at_d = torch.from_numpy(at).cuda()
        back = torch.from_numpy(rp[at].astype(np.int64)).cuda()[:, None] - torch.arange(c.lengths[s], device="cuda")
        see = back >= 0
        if anc is not None:
            see &= (back > 63) | (((anc[at_d, None] >> back.clamp(0, 63)) & 1) == 1)
        yield s, at_d, see


def attend(c, q, rs, rp, anc=None):
    """out, lse (float64) and what each may be off by."""
    rows, G = len(rs), c.hq // c.hkv
    out, tol = (torch.zeros(rows, c.hq, 128, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, ltol = (torch.zeros(rows, c.hq, dtype=torch.float64, device="cuda") for _ in range(2))
    for s, at, see in _rows(c, rs, rp, anc):
        for g in range(c.hkv):
            K, V = c.values(s, 0, g), c.values(s, 1, g)
            for h in range(g * G, (g + 1) * G):
                Q = q[at, h].double()
                x = torch.where(see, SCALE * (Q @ K.T), -torch.inf)
                xa = torch.where(see, SCALE * (Q.abs() @ K.abs().T), 0.0).amax(-1, keepdim=True)
                m = x.amax(-1, keepdim=True)
                e = (x - m).exp()
                z = e.sum(-1, keepdim=True)
                es = 2 * 128 * U * xa + 2.0 ** -20
                out[at, h], lse[at, h] = e @ V / z, (m + z.log())[:, 0]
                a = e @ V.abs() / z
                tol[at, h] = (2.0 ** -8 * out[at, h].abs() + a * (2.0 ** -11 + 2 * es)
                              + c.lengths[s] * 2.0 ** -25 / z * V.abs().max() + 1e-30)
                ltol[at, h] = es[:, 0] + 4 * U * (lse[at, h].abs() + m[:, 0].abs() + 20)
    return out, lse, tol, ltol


def mass(c, q, lse, rs, rp, old, decay):
    """The sums and what each may be off by."""
    G = c.hq // c.hkv
    out, tol = old.double(), torch.zeros_like(old, dtype=torch.float64)
    for s, at, see in _rows(c, rs, rp, None):
        L = c.lengths[s]
        for g in range(c.hkv):
            K = c.values(s, 0, g)
            add, err = (torch.zeros(L, dtype=torch.float64, device="cuda") for _ in range(2))
            for h in range(g * G, (g + 1) * G):
                Q, l = q[at, h].double(), lse[at, h].double()[:, None]
                x = SCALE * (Q @ K.T)
                w = torch.where(see, (x - l).exp(), 0.0)
                add += w.sum(0)
                err += (w * (2 * 128 * U * SCALE * (Q.abs() @ K.abs().T) + 4 * U * (x.abs() + l.abs()) + 2.0 ** -20)).sum(0)
            n = len(at) * G + 2
            out[s, g, :L] = (decay * out[s, g, :L] if decay else 0) + add
            tol[s, g, :L] = err + n * U * (add + out[s, g, :L].abs()) + 1e-37
    return out, tol


def assert_within(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all(), what + ": not finite"
    bad = err > tol
    if bad.any():
        i = int((err / tol.clamp(min=1e-300)).flatten().argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {i}: got "
                             f"{got.flatten()[i].item()} ref {ref.flatten()[i].item()} allowed {tol.flatten()[i].item()}")
