"""tfpa_write_qkv of many rows on the GPU: the kernel whose warps take several heads at once (from 8,192 heads a launch
on) against the definition with its roundings, and against the same rows in smaller calls."""

import numpy as np
import pytest
import torch

from oracle import e4m3, fp4
from paged_kv_cache_235_gb300 import binding as B
from tests.test_gpu_qkv import Call

pytestmark = pytest.mark.gpu

WIDE = 8192                                       # heads of a launch


def stored_rows(c, w, rs, rp):
    """What the cache holds at every row of a call, [rows][hkv][..]: bf16 values, e4m3 bytes, or codes and scales."""
    parts = []
    for s in sorted(set(rs.tolist())):
        at = torch.from_numpy(rp[rs == s].astype(np.int64)).cuda()
        page = at // 256
        if s in c.slabs:
            x = c.slabs[s][w][:, page]                             # [hkv][rows][..]
            x = x.transpose(0, 1)
        else:
            x = (c.v_pool if w else c.k_pool)[c.segs[s].page_table.long()[page]]
        n = torch.arange(len(at), device="cuda")
        if c.kv != "fp4":
            parts.append(x[n, :, at % 256])
        else:
            h = x.reshape(len(at), c.hkv, 2, 9216)[n, :, at // 128 % 2]
            codes = h[..., :8192].unflatten(-1, (128, 64))[n, :, at % 128]
            scales = h[..., 8192:].unflatten(-1, (128, 8))[n, :, at % 128]
            parts.append(torch.cat([codes, scales], -1))
    return torch.cat(parts)


class Many(Call):
    """A call whose row tables are in the order of the streams."""

    def heads(self):
        return len(self.rs) * (self.c.hq + self.c.hkv)

    def units(self):
        """Steps of a launch: eight q heads, or four kv heads, of a row."""
        return len(self.rs) * (-(-self.c.hq // 8) + -(-self.c.hkv // 4))

    def launches(self):
        with B.record_launches() as rec:
            B.tfpa_write_qkv(self.c.cache, self.c.segs, self.q, self.k, self.v, self.q_out[1:-1], self.rs, self.rp, stream=0, **self.kw)
        return rec

    def bytes_of(self, y, w):
        """float32 rows [rows][hkv][128] as the cache has to hold them."""
        c = self.c
        if c.kv == "bf16":
            return torch.from_numpy(y).to(torch.bfloat16).view(torch.int16)
        out = []
        for g in range(c.hkv):
            sc = np.float32((c.v_scale if w else c.k_scale)[g].item())
            x = np.ascontiguousarray(y[:, g])
            out.append(e4m3.quantise(x, sc) if c.kv == "fp8" else np.concatenate(fp4.quantise(x, sc), -1))
        return torch.from_numpy(np.stack(out, 1).astype(np.uint8))

    def check_all(self, out, rows=None, q_rows=None):
        at = torch.arange(len(self.rs)) if rows is None else torch.as_tensor(rows)
        qa = at if q_rows is None else torch.as_tensor(q_rows)
        q = torch.from_numpy(self.expected(self.q, "q_weight")).to(torch.bfloat16)
        assert torch.equal(out.cpu().view(torch.int16)[qa], q.view(torch.int16)[qa])
        for w, y in ((0, self.expected(self.k, "k_weight")), (1, self.v.float().cpu().numpy())):
            got = stored_rows(self.c, w, self.rs, self.rp).cpu()
            got = got.view(torch.int16) if self.c.kv == "bf16" else got
            want = self.bytes_of(y, w)
            bad = (got[at] != want[at]).flatten(1).any(1)
            assert not bad.any(), (w, at[bad][:5])

    def everything(self):
        c = self.c
        return [c.k_pool, c.v_pool, *[x for p in c.slabs.values() for x in p]]


BIG = dict(counts=(600, 1, 400), lengths=(700, 257, 900))
SHAPES = [dict(BIG), dict(BIG, norm=False, rot=0), dict(BIG, norm=False, inter=True), dict(BIG, rot=96, device_pos=True),
          dict(BIG, rot=64, inter=True), dict(BIG, rot=16, inter=True, device_pos=True), dict(BIG, rot=0, fused=False),
          dict(hq=5, hkv=5, rot=48, counts=(600, 0, 300), lengths=(700, 1, 900)),
          dict(hq=20, hkv=1, rot=112, inter=True, counts=(150, 9, 300), lengths=(700, 257, 900)),
          dict(hq=32, hkv=8, counts=(0, 170, 700), lengths=(1, 257, 900)),
          dict(hq=6, hkv=3, rot=32, counts=(1000, 200, 1500), lengths=(1100, 257, 1600))]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("kw", SHAPES, ids=range(len(SHAPES)))
def test_many_rows(kv, kw):
    call = Many(kv, **kw)
    assert call.heads() >= WIDE
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rec = call.launches()                                          # one warp a unit, or as many as the GPU holds
    assert [(r["items"], r["grid"]) for r in rec] == [(call.heads(), min(call.units(), 16 * sms))]
    before = [t.clone() for t in call.everything()]
    out = call.run()
    call.check_all(out)
    assert (call.q_out[[0, -1]] == 9).all() and int(call.c.err.item()) == 0
    # the same rows, fewer than 8,192 heads a call, into the cache as it was: every byte of it and of q
    after, q = [t.clone() for t in call.everything()], out.clone()
    for t, b in zip(call.everything(), before):
        t.copy_(b)
    out.fill_(9)
    step = (WIDE - 1) // (call.c.hq + call.c.hkv)
    kwargs = {k: v for k, v in call.kw.items() if k != "rope_pos"}
    for i in range(0, len(call.rs), step):
        sl = slice(i, i + step)
        pos = call.kw.get("rope_pos")
        B.tfpa_write_qkv(call.c.cache, call.c.segs, call.q[sl], call.k[sl], call.v[sl], out[sl], call.rs[sl], call.rp[sl],
                         rope_pos=None if pos is None else pos[sl], **kwargs)
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(call.everything(), after))


def test_runs_that_change_within_a_warps_rows():
    """Sixty streams of 3 to 40 rows, so that a warp's equal run of rows crosses them."""
    rng = np.random.default_rng(7)
    counts = [int(n) for n in rng.integers(3, 41, 60)]
    lengths = [n + int(x) for n, x in zip(counts, rng.integers(0, 300, 60))]
    call = Many("fp8", hq=16, hkv=4, counts=counts, lengths=lengths, paged=[i % 3 != 1 for i in range(60)], rot=64, inter=True)
    assert call.heads() >= WIDE and len(call.launches()) == 1
    call.check_all(call.run())


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_many_rows_with_positions_off_the_table(kv):
    call = Many(kv, **BIG, device_pos=True)
    bad = np.array([0, 1, 2, 303, 304, 599, 600, 700, 1000])
    call.kw["rope_pos"][torch.from_numpy(bad).cuda()] = torch.tensor([-1, call.kw["rope_cos"].shape[0], 2**31 - 1] * 3, dtype=torch.int32,
                                                                     device="cuda")
    held = [stored_rows(call.c, w, call.rs, call.rp).clone() for w in (0, 1)]
    out = call.run()
    good = np.setdiff1d(np.arange(len(call.rs)), bad)
    assert int(call.c.err.item()) == 4 and (out[torch.from_numpy(bad).cuda()] == 9).all()
    for w in (0, 1):
        now = stored_rows(call.c, w, call.rs, call.rp)
        assert torch.equal(now[bad].view(torch.uint8), held[w][bad].view(torch.uint8))
    call.kw["rope_pos"][torch.from_numpy(bad).cuda()] = 0
    call.check_all(out, good)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_many_rows_with_a_page_out_of_range(kv):
    """The rows on it keep their place's bytes; their q is handed out all the same."""
    call = Many(kv, **BIG)
    table = call.c.segs[2].page_table
    page = int(table[2])                              # positions 512 .. 767 of stream 2
    bad = np.flatnonzero((call.rs == 2) & (call.rp // 256 == 2))
    assert len(bad) == 256
    held = [stored_rows(call.c, w, call.rs, call.rp).clone() for w in (0, 1)]
    before = [t.clone() for t in call.everything()]
    for id_ in (call.c.num_pages, -1):
        for t, b in zip(call.everything(), before):
            t.copy_(b)
        call.c.err.zero_()
        table[2] = id_
        out = call.run()
        table[2] = page
        assert int(call.c.err.item()) == 1
        for w in (0, 1):
            now = stored_rows(call.c, w, call.rs, call.rp)
            assert torch.equal(now[bad].view(torch.uint8), held[w][bad].view(torch.uint8))
        call.check_all(out, np.setdiff1d(np.arange(len(call.rs)), bad), np.arange(len(call.rs)))


def test_many_rows_in_place():
    call = Many("fp8", **BIG, fused=False)
    call.q = call.q.contiguous()
    want = call.run().clone()
    assert torch.equal(call.run(q_out=call.q), want)


def test_many_rows_of_keys_and_values_only():
    call = Many("fp4", hq=8, hkv=8, counts=(700, 20, 400), lengths=(700, 257, 900))
    assert len(call.rs) * 8 >= WIDE
    B.tfpa_write_qkv(call.c.cache, call.c.segs, None, call.k, call.v, None, call.rs, call.rp, **call.kw)
    for w, y in ((0, call.expected(call.k, "k_weight")), (1, call.v.float().cpu().numpy())):
        assert torch.equal(stored_rows(call.c, w, call.rs, call.rp).cpu(), call.bytes_of(y, w))
    assert (call.q_out == 9).all()
