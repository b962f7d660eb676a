"""Rotary tables and a projection's rows on the GPU: tables against the formula in 64 bits, q and the stored bytes
against the definition with its roundings, and against the formula in 64 bits."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import e4m3, fp4
from paged_kv_cache_235_gb300 import binding as B
from tests.gpu64 import LongCase, last_rows

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                   # half a float32 step
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def freqs(s):
    """The table's frequencies, as the header defines them."""
    r, f = s.rot_dim, s.factor
    base = s.base * f ** (r / (r - 2)) if s.scaling == "base" else s.base
    w = base ** (-2.0 * np.arange(r // 2) / r)
    if s.scaling == "linear":
        return w / f
    if s.scaling == "bands":
        u = np.clip((s.orig_len * w / (2 * math.pi) - s.low) / (s.high - s.low), 0, 1)
        return w * u + w / f * (1 - u)
    if s.scaling == "ramp":
        dim = lambda n: r * math.log(s.orig_len / (2 * math.pi * n)) / (2 * math.log(s.base))  # noqa: E731
        a, b = max(math.floor(dim(s.high)), 0), min(math.ceil(dim(s.low)), r - 1)
        u = np.clip(1 - (np.arange(r // 2) - a) / max(b - a, 0.001), 0, 1)
        return w * u + w / f * (1 - u)
    return w


@pytest.mark.parametrize("first,n", [(0, 1), (0, 300), (131072, 257), (2**24 - 3, 7), (2**31 - 5, 5)])
@pytest.mark.parametrize("kw", [
    dict(base=1e4), dict(base=5e5, rot_dim=16), dict(base=1e4, rot_dim=96, scaling="linear", factor=3.7),
    dict(base=1e6, rot_dim=64, scaling="base", factor=8.0), dict(base=5e5, scaling="bands", factor=8.0, orig_len=8192, low=1.0, high=4.0),
    dict(base=1e4, scaling="ramp", factor=16.0, orig_len=4096, low=1.0, high=32.0, attn_scale=1.277),
    dict(base=1e4, rot_dim=32, scaling="ramp", factor=2.0, orig_len=1, low=1.0, high=32.0)])
def test_tables(kw, first, n):
    s = B.RopeSpec(**kw)
    half = s.rot_dim // 2
    c, d = (torch.full((n + 2, half), 7.0, device="cuda") for _ in range(2))
    B.tfpa_rope_table(s, first, c[1:n + 1], d[1:n + 1])
    assert (c[[0, -1]] == 7).all() and (d[[0, -1]] == 7).all()
    w = freqs(s)
    frac = np.array([[float(((first + t) * Fraction(float(f)) / TWO_PI) % 1) for f in w] for t in range(n)])
    ang = 2 * math.pi * frac
    # the fraction of a turn is right to t 2^-65; it is rounded to float32 within an eighth of a turn, and the sine, its
    # factor, and the product take a few roundings; two roundings of a power's frequency (none of 1) move a far angle
    tol = s.attn_scale * (6 * U + (first + n) * (2.0 ** -62 + np.where(w == 1, 0, w * 2.0 ** -51)))[None]
    for got, ref in ((c, np.cos(ang)), (d, np.sin(ang))):
        err = np.abs(got[1:n + 1].double().cpu().numpy() - s.attn_scale * ref)
        assert (err <= tol).all(), float((err / tol).max())


# ---------------------------------------------------------------- rows
def norm32(x, w, eps):
    sq = x * x
    while sq.shape[-1] > 1:
        sq = sq[..., 0::2] + sq[..., 1::2]
    return x * (np.float32(1) / np.sqrt(sq / np.float32(128) + np.float32(eps))) * w


def turn32(x, cos, sin, pos, inter):
    h = cos.shape[1]
    i = 2 * np.arange(h) if inter else np.arange(h)
    j = i + (1 if inter else h)
    c, s = cos[pos][:, None], sin[pos][:, None]
    y = x.copy()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
    return y


def stored(c, s, w, pos):
    """What the cache holds at position pos of stream s, every kv head: bf16 values, e4m3 bytes, or (codes, scales)."""
    page = c._page(s, w, pos // 256)
    if c.kv != "fp4":
        return page[:, pos % 256]
    h = page.view(c.hkv, 2, 9216)[:, (pos % 256) // 128]
    return h[:, :8192].reshape(c.hkv, 128, 64)[:, pos % 128], h[:, 8192:].reshape(c.hkv, 128, 8)[:, pos % 128]


class Call:
    """A call of tfpa_write_qkv and what it has to leave behind."""

    def __init__(self, kv, hq=8, hkv=2, counts=(3, 1, 5), lengths=(300, 257, 900), paged=(True, False, True), norm=True, rot=128, inter=False,
                 device_pos=False, eps=1e-6, fused=True, seed=5, scale=1.0):
        self.c = c = LongCase(kv, lengths, paged, hq, hkv, seed)
        self.rs, self.rp = last_rows(lengths, counts)
        rows = len(self.rs)
        g = c.g
        heads = hq + 2 * hkv
        x = (torch.randn(rows, heads + (0 if fused else 3), 128, generator=g, device="cuda") * scale).to(torch.bfloat16)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:heads]
        if not fused:
            self.k, self.v = self.k.clone(), self.v.clone()
        self.x = x
        self.kw = dict(eps=eps)
        if norm:
            self.kw.update(q_weight=1 + 0.3 * torch.randn(128, generator=g, device="cuda"), k_weight=1 + 0.3 * torch.randn(128, generator=g, device="cuda"))
        if rot:
            n = max(lengths) + 9
            a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * (1e4 ** (-2 * torch.arange(rot // 2, device="cuda") / rot))
            self.kw.update(rope_cos=a.cos().float(), rope_sin=a.sin().float(), interleaved=inter)
            if device_pos:
                self.kw["rope_pos"] = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
        self.q_out = torch.full((rows + 2, hq, 128), 9.0, dtype=torch.bfloat16, device="cuda")

    def run(self, q_out=None, **kw):
        out = self.q_out[1:-1] if q_out is None else q_out
        B.tfpa_write_qkv(self.c.cache, self.c.segs, self.q, self.k, self.v, out, self.rs, self.rp, **{**self.kw, **kw})
        torch.cuda.synchronize()
        return out

    def expected(self, x, weight):
        """float32 heads after norm and rotation, every step rounded."""
        y = x.float().cpu().numpy()
        if weight in self.kw:
            y = norm32(y, self.kw[weight].cpu().numpy(), self.kw["eps"])
        if "rope_cos" in self.kw:
            pos = self.rp if self.kw.get("rope_pos") is None else self.kw["rope_pos"].cpu().numpy()
            y = turn32(y, self.kw["rope_cos"].cpu().numpy(), self.kw["rope_sin"].cpu().numpy(), pos, self.kw["interleaved"])
        return y

    def check(self, out, rows=None):
        c = self.c
        q = torch.from_numpy(self.expected(self.q, "q_weight")).to(torch.bfloat16)
        rows = range(len(self.rs)) if rows is None else rows
        at = torch.tensor(list(rows), dtype=torch.long)
        assert torch.equal(out.cpu().view(torch.int16)[at], q.view(torch.int16)[at])
        for w, y, sc in ((0, self.expected(self.k, "k_weight"), c.k_scale), (1, self.v.float().cpu().numpy(), c.v_scale)):
            for r in rows:
                got = stored(c, int(self.rs[r]), w, int(self.rp[r]))
                if c.kv == "bf16":
                    assert torch.equal(got.cpu().view(torch.int16), torch.from_numpy(y[r]).to(torch.bfloat16).view(torch.int16)), (w, r)
                    continue
                for g in range(c.hkv):
                    if c.kv == "fp8":
                        assert np.array_equal(got[g].cpu().numpy(), e4m3.quantise(y[r, g], np.float32(sc[g].item()))), (w, r, g)
                    else:
                        codes, scales = fp4.quantise(y[r, g], np.float32(sc[g].item()))
                        assert np.array_equal(got[0][g].cpu().numpy(), codes) and np.array_equal(got[1][g].cpu().numpy(), scales), (w, r, g)

    def snapshot(self):
        c = self.c
        return [t.clone() for t in (c.k_pool, c.v_pool, *[x for p in c.slabs.values() for x in p])]

    def untouched(self, before, but=()):
        """Nothing but the call's rows (those in `but`: not even they) has changed."""
        c = self.c
        after = [c.k_pool, c.v_pool, *[x for p in c.slabs.values() for x in p]]
        saved = [t.clone() for t in after]
        self_rows = [(int(s), int(p)) for r, (s, p) in enumerate(zip(self.rs, self.rp)) if r not in but]
        now = [(w, s, p, stored(c, s, w, p)) for s, p in self_rows for w in (0, 1)]
        keep = [tuple(x.clone() for x in (v if isinstance(v, tuple) else (v,))) for *_, v in now]
        for t, b in zip(after, before):
            t.copy_(b)                               # the old state, then the rows put back: what the call should have left
        for (w, s, p, _), v in zip(now, keep):
            for dst, src in zip(stored(c, s, w, p) if isinstance(stored(c, s, w, p), tuple) else (stored(c, s, w, p),), v):
                dst.copy_(src)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(after, saved))


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("kw", [
    dict(), dict(norm=False, rot=0), dict(norm=False, inter=True), dict(rot=96, device_pos=True), dict(rot=64, inter=True), dict(rot=16),
    dict(rot=16, inter=True, device_pos=True), dict(rot=0, fused=False), dict(hq=5, hkv=5, rot=48), dict(hq=20, hkv=1, rot=112, inter=True),
    dict(hq=32, hkv=2, counts=(0, 0, 70), lengths=(1, 1, 200))])
def test_rows(kv, kw):
    call = Call(kv, **kw)
    before = call.snapshot()
    out = call.run()
    call.check(out)
    call.untouched(before)
    assert (call.q_out[[0, -1]] == 9).all() and int(call.c.err.item()) == 0


@pytest.mark.parametrize("scale", [1.0, 1e-18, 1e18])
def test_q_against_the_formula_in_64_bits(scale):
    call = Call("bf16", scale=scale, eps=1e-12)
    out = call.run().double().cpu().numpy()
    x = call.q.double().cpu().numpy()
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(1e-12))) * call.kw["q_weight"].double().cpu().numpy()
    if scale == 1e18:                                # squares of 1e36 add up to 1e38: still within float32
        assert np.isfinite(y).all()
    c, s = (call.kw[n].double().cpu().numpy()[call.rp][:, None] for n in ("rope_cos", "rope_sin"))
    a, b = y[..., :64], y[..., 64:]
    ref = np.concatenate([a * c - b * s, b * c + a * s], -1)
    size = np.concatenate([np.abs(a * c) + np.abs(b * s)] * 2, -1) + np.abs(ref)
    # a sum of 128 squares in 7 levels, root, quotient, two products; then product and sum: at most 20 roundings in all;
    # squares below the smallest normal (a scale of 1e-18) lose 2^-150 each, next to eps
    assert (np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + size * (20 * U + 2.0 ** -149 * 128 / 1e-12) + 1e-38).all()


def test_large_call_crosses_launches_and_types():
    call = Call("fp4", counts=(2900, 40, 3001), lengths=(2905, 45, 3010), hq=8, hkv=2)
    order = np.random.default_rng(1).permutation(len(call.rs))[:700]
    call.rs, call.rp = call.rs[order], call.rp[order]                  # hundreds of single rows: several launches
    call.q, call.k, call.v = (t[:700] for t in (call.q, call.k, call.v))
    call.q_out = call.q_out[:702]
    before = call.snapshot()
    out = call.run()
    call.check(out)
    call.untouched(before)


def test_q_in_place():
    call = Call("fp8", fused=False)
    call.q = call.q.contiguous()
    want = call.run().clone()
    assert torch.equal(call.run(q_out=call.q), want)


def test_kv_only_and_empty():
    call = Call("bf16")
    B.tfpa_write_qkv(call.c.cache, call.c.segs, None, call.k, call.v, None, call.rs, call.rp, **call.kw)
    out = call.q_out[1:-1]
    ref = Call("bf16")
    ref.run()
    for a, b in ((call.c.k_pool, ref.c.k_pool), (call.c.v_pool, ref.c.v_pool), (call.c.slabs[1][0], ref.c.slabs[1][0])):
        assert bool((a.view(torch.int16) == b.view(torch.int16)).all())       # the bits: NaN lies behind the streams' ends
    assert bool((out == 9).all())
    e = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    B.tfpa_write_qkv(call.c.cache, call.c.segs, e, e[:, :2], e[:, :2], e, [], [])


def test_rotary_position_outside_the_table_leaves_the_row_unwritten():
    call = Call("fp4", device_pos=True)
    call.kw["rope_pos"][2], call.kw["rope_pos"][4] = -1, call.kw["rope_cos"].shape[0]
    before = call.snapshot()
    out = call.run()
    good = [r for r in range(len(call.rs)) if r not in (2, 4)]
    assert (out[[2, 4]] == 9).all() and int(call.c.err.item()) == 4
    call.kw["rope_pos"][[2, 4]] = 0
    call.check(out, good)
    call.untouched(before, but=(2, 4))


def test_page_out_of_range_leaves_k_and_v_unwritten():
    call = Call("bf16", lengths=(300, 257, 900))
    table = call.c.segs[2].page_table
    page = int(table[3])                               # positions 768.. of stream 2: its rows of the call
    table[3] = call.c.num_pages
    before = call.snapshot()
    out = call.run()
    table[3] = page
    bad = [r for r in range(len(call.rs)) if call.rs[r] == 2]
    call.untouched(before, but=bad)
    call.check(out, [r for r in range(len(call.rs)) if r not in bad])
    assert int(call.c.err.item()) == 1
    q = torch.from_numpy(call.expected(call.q, "q_weight")).to(torch.bfloat16)
    assert torch.equal(out.cpu(), q)                   # q does not hang on the page


def test_special_values():
    """NaN and infinities go where the formula takes them; a zero head stays zero; a quantised store stays finite."""
    call = Call("fp4", norm=True, rot=64)
    x = call.x
    x[0, 0, 3], x[1, 1], x[2, 8, 5], x[3, 9, 100], x[4, 10, 7] = float("nan"), 0.0, float("nan"), float("inf"), float("-inf")
    with np.errstate(all="ignore"):
        out = call.run()
        q = torch.from_numpy(call.expected(call.q, "q_weight"))
    a, b = out.float().cpu(), q.to(torch.bfloat16).float()
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())
    assert torch.isnan(a[0, 0]).all() and (a[1, 1] == 0).all()
    k, v = (torch.empty(len(call.rs), 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.tfpa_read_kv(call.c.cache, call.c.segs, k, v, call.rs, call.rp)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_captured_on_a_stream_and_replayed_with_other_rows():
    call = Call("fp8")
    call.run()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.tfpa_write_qkv(call.c.cache, call.c.segs, call.q, call.k, call.v, call.q_out[1:-1], call.rs, call.rp, **call.kw)
    call.x.copy_(torch.randn_like(call.x.float()).to(torch.bfloat16))
    g.replay()
    torch.cuda.synchronize()
    call.check(call.q_out[1:-1])


def test_tables_feed_both_stores():
    """A full-head table serves tfpa_write_kv_rope too: the same K as tfpa_write_qkv without a norm."""
    call = Call("bf16", norm=False, rot=128)
    s = B.RopeSpec(5e5, scaling="linear", factor=4.0)
    cos, sin = (torch.empty(1000, 64, device="cuda") for _ in range(2))
    B.tfpa_rope_table(s, 0, cos, sin)
    call.run(rope_cos=cos, rope_sin=sin)
    k = call.c.k_pool.clone()
    call.c.k_pool.zero_()
    B.tfpa_write_kv_rope(call.c.cache, call.c.segs, call.k.contiguous(), call.v.contiguous(), call.rs, call.rp, cos, sin)
    for s_, p in zip(call.rs, call.rp):
        if s_ != 1:
            got = stored(call.c, int(s_), 0, int(p)).clone()
            call.c.k_pool, other = k, call.c.k_pool
            assert torch.equal(got, stored(call.c, int(s_), 0, int(p)))
            call.c.k_pool = other
