"""What is measured of the 4-bit cache and of cache eviction: four operators, their plain forms in
elementary torch operations, and their definitions in 64 bits.

store   new K / V rows quantised into a 4-bit cache (optionally K rotated first), and read back as the
        values that the cache holds: ``tfpa_write_kv``, ``tfpa_write_kv_rope``, ``tfpa_read_kv``
attend  attention over a cache held in 4 bits: single tokens, verify rows, draft trees, a decode step that
        stores its rows, prompt chunks: ``tfpa_decode``, ``tfpa_decode_tree``, ``tfpa_decode_append``,
        ``tfpa_prefill``
mass    the attention weight that each cached key got from a call's rows, accumulated per kv head:
        ``tfpa_key_mass``
evict   all but the keys of largest accumulated weight leave the cache, in place: ``tfpa_evict_kv``

The 4-bit cache: a page (256 positions) of one kv head is a block of two halves of 128 positions, each
[128][64] bytes of e2m1 codes (two head dims a byte, the even one in the low nibble) and then [128][8] e4m3
scales, one per 16 head dims.  A value is code * scale * k_scale[kv head].
"""

import math

import numpy as np
import torch

own = False

PAGE, D, HALF = 256, 128, 128
BLOCK = 2 * HALF * (D // 2 + D // 16)          # bytes of one page of one kv head, 4 bits
SCALE = 1.0 / math.sqrt(D)
SINK = 4


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decode step's new rows, one a stream: the smallest store
        dict(name="store_step", kind="store", hq=32, hkv=8, streams=8, lo=8192, hi=8192, rows=1, rope=False),
        # a prompt chunk's rows stored with their rotary positions
        dict(name="store_prompt_rope", kind="store", hq=32, hkv=8, streams=1, lo=32768, hi=32768, rows=4096, rope=True),
        # one short chat stream, one token: latency
        dict(name="decode_one_stream", kind="attend", form="decode", hq=8, hkv=2, streams=1, lo=1000, hi=1000, rows=1, slabs=0),
        # a serving batch, half in slabs and half in pages
        dict(name="decode_batch", kind="attend", form="decode", hq=32, hkv=8, streams=8, lo=8192, hi=8192, rows=1, slabs=4),
        # a serving batch of very different lengths; the step stores its rows itself
        dict(name="step_ragged", kind="attend", form="append", hq=32, hkv=8, streams=16, lo=1003, hi=109001, rows=1, slabs=0),
        # four draft rows verified on long streams
        dict(name="verify_long", kind="attend", form="decode", hq=32, hkv=8, streams=8, lo=65536, hi=65536, rows=4, slabs=0),
        # 16-node draft trees
        dict(name="tree_16", kind="attend", form="tree", hq=32, hkv=8, streams=8, lo=32761, hi=32761, rows=16, slabs=0),
        # a prompt chunk over a long prefix
        dict(name="prompt_chunk", kind="attend", form="prefill", hq=32, hkv=8, streams=1, lo=32768, hi=32768, rows=4096, slabs=0),
        # weight accumulated at every decode step, bf16 cache
        dict(name="mass_step", kind="mass", dtype="bf16", hq=32, hkv=8, streams=8, lo=8192, hi=8192, rows=1, decay=1.0),
        # weight that a prompt's last rows give, 4-bit cache
        dict(name="mass_window", kind="mass", dtype="fp4", hq=32, hkv=8, streams=4, lo=32001, hi=65001, rows=32, decay=0.95),
        # a short stream cut to half; the next token then attends to what is left
        dict(name="evict_one_stream", kind="evict", dtype="fp4", hq=8, hkv=2, streams=1, lo=1001, hi=1001, share=0.5, recent=64),
        # a batch of long streams cut to half
        dict(name="evict_batch", kind="evict", dtype="bf16", hq=32, hkv=8, streams=8, lo=32768, hi=65536, share=0.5, recent=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["store", "attend", "attend", "attend", "mass", "evict"])
    hq, hkv = rng.choice([(8, 2), (32, 8), (16, 4), (10, 2), (8, 8), (6, 1), (24, 8)])
    c = dict(kind=kind, hq=hq, hkv=hkv)
    if kind == "store":
        streams = rng.randint(1, 8)
        rows = _log(rng, 1, 4096 // streams)
        lo = rows + _log(rng, 1, 4096)
        return dict(c, streams=streams, lo=lo, hi=lo + _log(rng, 1, 24000), rows=rows, rope=rng.random() < 0.5)
    if kind == "attend":
        form = rng.choice(["decode", "decode", "append", "tree", "prefill"])
        if form == "prefill":
            rows = _log(rng, 2, 2048)
            lo = rows + _log(rng, 1, 16384)
            return dict(c, form=form, streams=1, lo=lo, hi=lo, rows=rows, slabs=rng.randint(0, 1))
        streams = _log(rng, 1, 16)
        rows = {"decode": rng.choice([1, 1, 2, 3, 4, 7]), "append": rng.choice([1, 1, 2]), "tree": rng.randint(2, 24)}[form]
        lo = rows + _log(rng, 1, 8000)
        hi = max(lo, _log(rng, 256, 200000 // streams))
        return dict(c, form=form, streams=streams, lo=lo, hi=hi, rows=rows, slabs=0 if form == "append" else rng.randint(0, min(3, streams)))
    dtype = rng.choice(["bf16", "fp8", "fp4"])
    streams = _log(rng, 1, 8)
    if kind == "mass":
        rows = _log(rng, 1, 48)
        lo = rows + _log(rng, 1, 8000)
        hi = max(lo, _log(rng, 256, 120000 // streams))
        return dict(c, dtype=dtype, streams=streams, lo=lo, hi=hi, rows=rows, decay=rng.choice([0.0, 0.5, 0.95, 1.0]))
    lo = _log(rng, 300, 8000)
    hi = max(lo, _log(rng, 300, 120000 // streams))
    return dict(c, dtype=dtype, streams=streams, lo=lo, hi=hi, share=round(rng.uniform(0.3, 0.95), 2), recent=rng.choice([0, 1, 32, 64]))


def _lengths(c):
    """The streams' lengths: from lo to hi (one stream: hi), evenly over the logarithm."""
    n = c["streams"]
    return [int(round(c["hi"] * (c["lo"] / c["hi"]) ** (i / max(1, n - 1)))) for i in range(n)][::-1]


def _keep(c):
    return [max(SINK + c["recent"], min(L, int(L * c["share"]))) if L > SINK + c["recent"] else L for L in _lengths(c)]


def _row_bytes(dtype):
    return {"bf16": 2 * D, "fp8": D, "fp4": D // 2 + D // 16}[dtype]


def work(case):
    c, Ls = case, _lengths(case)
    hq, hkv = c["hq"], c["hkv"]
    if c["kind"] == "store":
        n = c["streams"] * c["rows"] * hkv * 2
        return {"bytes": n * (2 * (2 * D) + 2 * _row_bytes("fp4")), "flops": n * D * 8}
    if c["kind"] == "attend":
        rows = c["rows"] * len(Ls)
        pairs = sum(c["rows"] * L - c["rows"] * (c["rows"] - 1) // 2 for L in Ls)
        b = 2 * hkv * sum(Ls) * _row_bytes("fp4") + rows * hq * (4 * D + 4)
        return {"bytes": b, "flops": 4 * D * hq * pairs}
    if c["kind"] == "mass":
        rows = c["rows"] * len(Ls)
        pairs = sum(c["rows"] * L - c["rows"] * (c["rows"] - 1) // 2 for L in Ls)
        b = hkv * sum(Ls) * (_row_bytes(c["dtype"]) + (8 if c["decay"] else 4)) + rows * hq * (2 * D + 4)
        return {"bytes": b, "flops": 2 * D * hq * pairs}
    b = 0
    for L, n in zip(Ls, _keep(c)):
        moves = n * (L - n) / L                                   # survivors behind the cut, on average
        b += hkv * (8 * L + 4 * (L - n) + moves * (2 * 2 * _row_bytes(c["dtype"]) + 16))
    return {"bytes": b, "flops": hkv * sum(Ls) * 4}


# ------------------------------------------------------------------------------------------------ inputs
def _values(g, *shape):
    """K or V as a model writes them: normal, a few head dims several times larger."""
    x = torch.randn(*shape, generator=g, device="cuda")
    big = 1 + 4 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.06)
    return (x * big).to(torch.bfloat16)


def _e2m1_code(y):
    """Nearest e2m1 code (ties to the even code, saturating) of float32 y."""
    a = y.abs()
    mag = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return mag.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)


def _quantise(x, g):
    """x float32 [..., 128], g float32 [...]: codes [..., 64] uint8 and scales [..., 8] e4m3."""
    x = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf)
    b = x.unflatten(-1, (D // 16, 16))
    s = (b.abs().amax(-1) / (g * 6.0).unsqueeze(-1)).clamp(max=448.0).to(torch.float8_e4m3fn)
    step = s.float() * g.unsqueeze(-1)
    y = torch.where(step.unsqueeze(-1) > 0, b / step.unsqueeze(-1), torch.zeros((), device=x.device)).flatten(-2)
    code = _e2m1_code(y)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _pages(c):
    return max(-(-L // PAGE) for L in _lengths(c))


def _cache(c, g, dtype, slabs=0):
    """A filled cache in its stored form: pools with the streams in pages dealt from a permutation,
    the first `slabs` streams in slabs, scales per kv head, page tables."""
    S, hkv, P = c["streams"], c["hkv"], _pages(c)
    paged = S - slabs
    num_pages = max(1, paged * P + 3)
    perm = torch.randperm(num_pages, generator=g, device="cuda")[: paged * P].view(paged, P)
    st = dict(num_pages=num_pages, table=perm.to(torch.int32).contiguous(), slabs=slabs)
    for w in ("k", "v"):
        x = _values(g, S, hkv, P * PAGE, D)
        if dtype == "bf16":
            rows = x.view(S, hkv, P, PAGE, D)
            st[w + "_scale"] = None
            pool = torch.randn(num_pages, hkv, PAGE, D, generator=g, device="cuda").to(torch.bfloat16)
        else:
            amax = x.abs().amax(dim=(0, 2, 3)).float()
            st[w + "_scale"] = (amax / (448.0 if dtype == "fp8" else 2688.0)).contiguous()
            sc = st[w + "_scale"].view(1, hkv, 1)
            if dtype == "fp8":
                rows = (x.float() / sc.unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                rows = rows.view(S, hkv, P, PAGE, D)
                pool = torch.zeros(num_pages, hkv, PAGE, D, device="cuda", dtype=torch.float8_e4m3fn)
            else:
                code, s = _quantise(x.float(), sc)
                rows = torch.cat([code.view(S, hkv, P, 2, HALF * (D // 2)),
                                  s.view(torch.uint8).view(S, hkv, P, 2, HALF * (D // 16))], -1)
                rows = rows.view(S, hkv, P, BLOCK)
                pool = torch.randint(0, 256, (num_pages, hkv, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
        raw = pool.view(torch.uint8) if dtype == "fp8" else pool
        raw[perm.flatten()] = (rows.view(torch.uint8) if dtype == "fp8" else rows)[slabs:].transpose(1, 2).flatten(0, 1)
        st[w + "_pool"] = pool
        st[w + "_slab"] = rows[:slabs].contiguous() if slabs else None
        del x
    return st


def _rows_of(c):
    """Row tables: each stream's last `rows` positions."""
    Ls, R = _lengths(c), c["rows"]
    seg = np.repeat(np.arange(len(Ls), dtype=np.int32), R)
    pos = np.concatenate([np.arange(L - R, L, dtype=np.int32) for L in Ls])
    return seg, pos


def _tree_masks(n, rng):
    """Ancestor masks of a random draft tree of n nodes at consecutive positions: bit d of node i's mask
    says whether it sees the key d positions back."""
    par = [-1] + [int(rng.integers(0, i)) for i in range(1, n)]
    out = []
    for i in range(n):
        m, a = ((1 << 64) - 1) & ~((1 << (i + 1)) - 1), i
        while a >= 0:
            m |= 1 << (i - a)
            a = par[a]
        out.append(m)
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    rng = np.random.default_rng(int(seed) + 5)
    hq, hkv, Ls = c["hq"], c["hkv"], _lengths(c)
    S = len(Ls)
    st = dict(c=c, lengths=Ls)
    if c["kind"] == "evict":
        st.update(_cache(c, g, c["dtype"]))
        cap = _pages(c) * PAGE
        n = torch.tensor(Ls, device="cuda").view(S, 1, 1)
        slot = torch.arange(cap, device="cuda").view(1, 1, cap)
        mass = torch.exp(2 * torch.randn(S, hkv, cap, generator=g, device="cuda"))
        mass = mass * (torch.rand(S, hkv, cap, generator=g, device="cuda") > 0.05)
        # positions of the slots' keys after earlier evictions: gaps, the older three quarters out of order
        gap = torch.randint(1, 3, (S, hkv, cap), generator=g, device="cuda")
        back = torch.where(slot < n, gap, 0).flip(-1).cumsum(-1).flip(-1)
        pos = 2 * n - back
        key = torch.where(slot < 3 * n // 4, torch.rand(S, hkv, cap, generator=g, device="cuda"), 2.0 + slot)
        pos = pos.gather(-1, key.argsort(-1))
        pos = torch.where(slot < SINK, slot, pos)
        st["mass0"] = torch.where(slot < n, mass, 0).contiguous()
        st["pos0"] = torch.where(slot < n, pos, -1).to(torch.int32).contiguous()
        st["mass"], st["key_pos"] = torch.empty_like(st["mass0"]), torch.empty_like(st["pos0"])
        st["keep"], st["next_pos"] = np.array(_keep(c), np.int32), np.array([2 * L for L in Ls], np.int32)
        st["moves"] = torch.zeros(S, hkv, cap + 4, device="cuda", dtype=torch.int32)
        if c["dtype"] == "fp4":
            st["q"] = torch.randn(S, hq, D, generator=g, device="cuda").to(torch.bfloat16)
            st["row_seg"], st["row_pos"] = np.arange(S, dtype=np.int32), st["keep"] - 1
            st["out"] = torch.empty(S, hq, D, device="cuda", dtype=torch.bfloat16)
            st["lse"] = torch.empty(S, hq, device="cuda")
        return st
    st["row_seg"], st["row_pos"] = _rows_of(c)
    rows = S * c["rows"]
    if c["kind"] == "store":
        st.update(_cache(dict(c, lo=1, hi=1), g, "fp4"))           # scales and a small cache ...
        P = _pages(c)
        st["num_pages"] = S * P + 3                                # ... then the streams' pages, unwritten
        st["table"] = torch.randperm(S * P + 3, generator=g, device="cuda")[: S * P].view(S, P).to(torch.int32)
        for w in ("k", "v"):
            st[w + "_pool"] = torch.randint(0, 256, (S * P + 3, hkv, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
            st[w + "_rows"] = _values(g, rows, hkv, D)
            st[w + "_scale"] = (st[w + "_rows"].abs().amax(dim=(0, 2)).float() / 2688.0 * 1.01).contiguous()
            st[w + "_back"] = torch.empty(rows, hkv, D, device="cuda", dtype=torch.bfloat16)
        if c["rope"]:
            t = torch.arange(max(Ls), device="cuda", dtype=torch.float64)[:, None]
            a = t * (1e6 ** (-2 * torch.arange(D // 2, device="cuda", dtype=torch.float64) / D))[None]
            st["cos"], st["sin"] = a.cos().float().contiguous(), a.sin().float().contiguous()
        return st
    st.update(_cache(c, g, c.get("dtype", "fp4"), c.get("slabs", 0)))
    st["q"] = torch.randn(rows, hq, D, generator=g, device="cuda").to(torch.bfloat16)
    if c["kind"] == "mass":
        st["lse"] = _attend(st, st["q"], want="lse")
        cap = _pages(c) * PAGE
        st["mass"] = torch.rand(S, hkv, cap, generator=g, device="cuda")
        return st
    st["out"] = torch.empty(rows, hq, D, device="cuda", dtype=torch.bfloat16)
    st["lse"] = torch.empty(rows, hq, device="cuda")
    if c["form"] == "tree":
        m = [v for _ in range(S) for v in _tree_masks(c["rows"], rng)]
        st["anc"] = torch.from_numpy(np.array(m, np.uint64).view(np.int64)).cuda()
    if c["form"] == "append":
        st["k_rows"], st["v_rows"] = _values(g, rows, hkv, D), _values(g, rows, hkv, D)
    return st


# ------------------------------------------------------------------------------------------------ plain forms
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _unpack(raw, scale_bytes, g):
    """Values (float32) of codes [..., 64] and scale bytes [..., 8], g broadcast over [...]."""
    lut = torch.tensor(_E2M1 + [-v for v in _E2M1], device=raw.device)
    two = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)          # [byte][low, high]
    x = two[raw.int()].flatten(-2)
    s = scale_bytes.contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(16, -1)
    return x * s * g.unsqueeze(-1)


def _halves(pool):
    """Codes and scales of a 4-bit pool [pages][hkv][BLOCK] as views [pages][hkv][2][128][..]."""
    h = pool.unflatten(-1, (2, BLOCK // 2))
    n = HALF * (D // 2)
    return h[..., :n].unflatten(-1, (HALF, D // 2)), h[..., n:].unflatten(-1, (HALF, D // 16))


def _dequant(st, w, dtype):
    """K or V of every stream, float32 [S][hkv][positions][128]."""
    blocks = st[w + "_pool"].view(torch.uint8)[st["table"].long()] if dtype == "fp8" else st[w + "_pool"][st["table"].long()]
    blocks = blocks.transpose(1, 2)                                              # [S'][hkv][P][...]
    if st["slabs"]:
        slab = st[w + "_slab"]
        blocks = torch.cat([slab.view(torch.uint8) if dtype == "fp8" else slab, blocks])
    if dtype == "bf16":
        return blocks.flatten(2, 3).float()
    g = st[w + "_scale"].view(1, -1, 1)
    if dtype == "fp8":
        return blocks.contiguous().view(torch.float8_e4m3fn).flatten(2, 3).float() * g.unsqueeze(-1)
    code, s = _halves(blocks)
    return _unpack(code.flatten(2, 4), s.flatten(2, 4), g)


def _scores(st, q, dtype):
    """Scaled and masked scores, float32 [S][hkv][rows * group][keys]."""
    c = st["c"]
    S, hkv, G = c["streams"], c["hkv"], c["hq"] // c["hkv"]
    R = q.shape[0] // S
    K = _dequant(st, "k", dtype)
    Q = q.float().view(S, R, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, hkv, R * G, D)
    s = (Q @ K.transpose(-1, -2)).mul_(SCALE)
    pos = torch.from_numpy(st["row_pos"].astype(np.int64)).cuda().view(S, R, 1)
    back = pos - torch.arange(K.shape[2], device="cuda").view(1, 1, -1)          # positions back
    hide = back < 0
    if "anc" in st:
        bit = (st["anc"].view(S, R, 1) >> back.clamp(0, 63)) & 1
        hide = hide | ((back < 64) & (bit == 0))
    hide = hide.repeat_interleave(G, 1).unsqueeze(1)
    return s.masked_fill_(hide, -math.inf)


def _attend(st, q, want="out"):
    c = st["c"]
    dtype = c.get("dtype", "fp4")
    S, hkv, G = c["streams"], c["hkv"], c["hq"] // c["hkv"]
    R = q.shape[0] // S
    s = _scores(st, q, dtype)
    m = s.amax(-1, keepdim=True)
    s.sub_(m).exp_()
    l = s.sum(-1, keepdim=True)
    lse = (m + l.log()).view(S, hkv, R, G).permute(0, 2, 1, 3).reshape(S * R, hkv * G)
    if want == "lse":
        return lse.contiguous()
    o = (s @ _dequant(st, "v", dtype)) / l
    o = o.view(S, hkv, R, G, D).permute(0, 2, 1, 3, 4).reshape(S * R, hkv * G, D)
    return o.to(torch.bfloat16), lse.contiguous()


def _place(st):
    """Page, half and row of each row of the call."""
    seg, pos = torch.from_numpy(st["row_seg"]).cuda().long(), torch.from_numpy(st["row_pos"]).cuda().long()
    return st["table"][seg, pos // PAGE].long(), (pos // HALF) % 2, pos % HALF


def _store(st, k, v):
    for w, x in (("k", k), ("v", v)):
        code, s = _quantise(x, st[w + "_scale"].view(1, -1).expand(x.shape[:2]))
        pid, half, r = _place(st)
        codes, scales = _halves(st[w + "_pool"])
        codes[pid, :, half, r] = code
        scales[pid, :, half, r] = s.view(torch.uint8)


def _rotate(st, k):
    pos = torch.from_numpy(st["row_pos"]).cuda().long()
    c, s = st["cos"][pos].unsqueeze(1), st["sin"][pos].unsqueeze(1)
    a, b = k[..., : D // 2], k[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def _plain_store(st):
    k, v = st["k_rows"].float(), st["v_rows"].float()
    _store(st, _rotate(st, k) if st["c"]["rope"] else k, v)
    out = []
    for w in ("k", "v"):
        pid, half, r = _place(st)
        codes, scales = _halves(st[w + "_pool"])
        out.append(_unpack(codes[pid, :, half, r], scales[pid, :, half, r], st[w + "_scale"].view(1, -1)).to(torch.bfloat16))
    return out


def _plain_mass(st):
    c = st["c"]
    S, hkv, G, R = c["streams"], c["hkv"], c["hq"] // c["hkv"], c["rows"]
    s = _scores(st, st["q"], c["dtype"])
    lse = st["lse"].view(S, R, hkv, G).permute(0, 2, 1, 3).reshape(S, hkv, R * G, 1)
    add = s.sub_(lse).exp_().sum(2)
    live = torch.arange(add.shape[-1], device="cuda").view(1, 1, -1) < torch.tensor(st["lengths"], device="cuda").view(S, 1, 1)
    old = st["mass"] * c["decay"] if c["decay"] else torch.zeros_like(st["mass"])
    st["mass"].copy_(torch.where(live, old + add, st["mass"]))
    return st["mass"]


def _plain_evict(st):
    c = st["c"]
    S, hkv = c["streams"], c["hkv"]
    st["mass"].copy_(st["mass0"])
    st["key_pos"].copy_(st["pos0"])
    mass, pos = st["mass"], st["key_pos"]
    cap = mass.shape[-1]
    slot = torch.arange(cap, device="cuda").view(1, 1, cap)
    n = torch.tensor(st["lengths"], device="cuda").view(S, 1, 1)
    keep = torch.from_numpy(st["keep"]).cuda().view(S, 1, 1)
    nxt = torch.from_numpy(st["next_pos"]).cuda().view(S, 1, 1)
    guarded = (pos < SINK) | (pos >= nxt - c["recent"])
    rank_key = torch.where(slot < n, torch.where(guarded, math.inf, mass), -math.inf)
    order = torch.sort(rank_key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order).contiguous())
    stays = rank < keep
    hole, mover = (slot < keep) & ~stays, (slot >= keep) & stays
    # the k-th mover's slot, and for each hole the slot of the mover that fills it
    kth = torch.sort((~mover).to(torch.uint8), dim=-1, stable=True).indices
    src = torch.where(hole, kth.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), slot)
    new_mass = torch.where(slot < keep, mass.gather(-1, src), torch.where(slot < n, 0.0, mass))
    new_pos = torch.where(slot < keep, pos.gather(-1, src), torch.where(slot < n, -1, pos))
    d_ = torch.arange(int(st["keep"].max()), device="cuda").view(1, 1, -1)         # every slot that is left takes its row
    f_ = src[..., : d_.shape[-1]]
    s_, g_ = torch.arange(S, device="cuda").view(S, 1, 1), torch.arange(hkv, device="cuda").view(1, hkv, 1)
    from_page, to_page = st["table"][s_, f_ // PAGE].long(), st["table"][s_, d_ // PAGE].long()
    for w in ("k", "v"):
        pool = st[w + "_pool"]
        if c["dtype"] == "fp4":
            for view in _halves(pool):
                view[to_page, g_, (d_ // HALF) % 2, d_ % HALF] = view[from_page, g_, (f_ // HALF) % 2, f_ % HALF]
        else:
            view = pool.view(torch.uint8) if c["dtype"] == "fp8" else pool
            view[to_page, g_, d_ % PAGE] = view[from_page, g_, f_ % PAGE]
    mass.copy_(new_mass)
    pos.copy_(new_pos)
    if c["dtype"] == "fp4":
        out, lse = _attend(st, st["q"])
        return {"mass": mass, "pos": pos, "out": out, "lse": lse}
    return {"mass": mass, "pos": pos, "k": st["k_pool"], "v": st["v_pool"]}


# ------------------------------------------------------------------------------------------------ the framework's calls
def _handles(st):
    """What a user's program keeps between calls: the cache, its segments, a scratch."""
    from paged_kv_cache_235_gb300 import binding as B
    if "cache" not in st:
        c = st["c"]
        dtype = c.get("dtype", "fp4")
        st["cache"] = B.Cache(dtype, c["hq"], c["hkv"], st["k_pool"], st["v_pool"], st["k_scale"], st["v_scale"], None, st["num_pages"])
        segs = []
        for i, L in enumerate(st["lengths"]):
            if i < st["slabs"]:
                segs.append(B.Seg(L, k_slab=st["k_slab"][i], v_slab=st["v_slab"][i], slab_cap=_pages(c) * PAGE))
            else:
                segs.append(B.Seg(L, page_table=st["table"][i - st["slabs"]]))
        st["segs"] = B.SegTable(segs)
        if c["kind"] == "evict":
            st["kept_segs"] = B.SegTable([B.Seg(int(n), page_table=st["table"][i]) for i, n in enumerate(st["keep"])])
        if "out" in st and c.get("form") != "prefill":
            st["scratch"] = B.make_scratch(min(128, len(st["row_seg"])), c["hq"])
    return B


def _own(st):
    B = _handles(st)
    c = st["c"]
    if c["kind"] == "store":
        if c["rope"]:
            B.tfpa_write_kv_rope(st["cache"], st["segs"], st["k_rows"], st["v_rows"], st["row_seg"], st["row_pos"], st["cos"], st["sin"])
        else:
            B.tfpa_write_kv(st["cache"], st["segs"], st["k_rows"], st["v_rows"], st["row_seg"], st["row_pos"])
        B.tfpa_read_kv(st["cache"], st["segs"], st["k_back"], st["v_back"], st["row_seg"], st["row_pos"])
        return [st["k_back"], st["v_back"]]
    if c["kind"] == "mass":
        B.tfpa_key_mass(st["cache"], st["segs"], st["q"], st["lse"], st["row_seg"], st["row_pos"], SCALE, st["mass"], decay=c["decay"])
        return st["mass"]
    if c["kind"] == "evict":
        st["mass"].copy_(st["mass0"])
        st["key_pos"].copy_(st["pos0"])
        B.tfpa_evict_kv(st["cache"], st["segs"], st["keep"], st["mass"], st["moves"], key_pos=st["key_pos"], next_pos=st["next_pos"],
                        sink=SINK, recent=c["recent"])
        if c["dtype"] == "fp4":
            B.tfpa_decode(st["cache"], st["kept_segs"], st["q"], st["row_seg"], st["row_pos"], SCALE, st["scratch"], st["out"], st["lse"])
            return {"mass": st["mass"], "pos": st["key_pos"], "out": st["out"], "lse": st["lse"]}
        return {"mass": st["mass"], "pos": st["key_pos"], "k": st["k_pool"], "v": st["v_pool"]}
    if c["form"] == "prefill":
        B.tfpa_prefill(st["cache"], st["segs"], st["q"], st["row_seg"], st["row_pos"], SCALE, st["out"], st["lse"])
    elif c["form"] == "tree":
        B.tfpa_decode_tree(st["cache"], st["segs"], st["q"], st["row_seg"], st["row_pos"], st["anc"], SCALE, st["scratch"], st["out"], st["lse"])
    elif c["form"] == "append":
        B.tfpa_decode_append(st["cache"], st["segs"], st["k_rows"], st["v_rows"], st["q"], st["row_seg"], st["row_pos"], SCALE, st["scratch"],
                             st["out"], st["lse"])
    else:
        B.tfpa_decode(st["cache"], st["segs"], st["q"], st["row_seg"], st["row_pos"], SCALE, st["scratch"], st["out"], st["lse"])
    return [st["out"], st["lse"]]


def run(state):
    if own:
        return _own(state)
    c = state["c"]
    if c["kind"] == "store":
        return _plain_store(state)
    if c["kind"] == "mass":
        return _plain_mass(state)
    if c["kind"] == "evict":
        return _plain_evict(state)
    if c["form"] == "append":
        _store(state, state["k_rows"].float(), state["v_rows"].float())
    return list(_attend(state, state["q"]))


# ------------------------------------------------------------------------------------------------ definitions in 64 bits
def _grid(bits_exp, bits_man, bias, top):
    """The non-negative values of a small float format, ascending."""
    vals = []
    for code in range(1 << (bits_exp + bits_man)):
        e, m = code >> bits_man, code & ((1 << bits_man) - 1)
        vals.append(m * 2.0 ** (1 - bias - bits_man) if e == 0 else (1 + m / 2.0 ** bits_man) * 2.0 ** (e - bias))
    return torch.tensor([v for v in vals if v <= top], dtype=torch.float64, device="cuda")


def _round_to(x, grid):
    """x >= 0 to the nearest value of the grid, ties to the even place, saturating."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    a, b = x - grid[lo], grid[hi] - x
    up = (b < a) | ((b == a) & (hi % 2 == 0))
    return torch.where(up, grid[hi], grid[lo])


def _exact_quantised(x, g):
    """x float64 [..., 128] as the 4-bit cache holds it."""
    e4m3, e2m1 = _grid(4, 3, 7, 448.0), _grid(2, 1, 1, 6.0)
    b = x.reshape(*x.shape[:-1], 8, 16)
    s = _round_to(b.abs().amax(-1, keepdim=True) / (6 * g[..., None, None]), e4m3)
    step = s * g[..., None, None]
    mag = _round_to(torch.where(step > 0, b.abs() / step, torch.zeros_like(b)), e2m1)
    return (torch.copysign(mag, b) * step).reshape(x.shape)


def _exact_head(st, w, i, h, n, dtype):
    """Stream i's first n keys or values of kv head h, float64 [n][128]."""
    P = -(-n // PAGE)
    if i < st["slabs"]:
        blocks = st[w + "_slab"][i, h, :P]
    else:
        blocks = st[w + "_pool"].view(torch.uint8 if dtype == "fp8" else st[w + "_pool"].dtype)[st["table"][i - st["slabs"], :P].long(), h]
    if dtype == "bf16":
        return blocks.reshape(P * PAGE, D)[:n].double()
    g = st[w + "_scale"][h].double()
    if dtype == "fp8":
        return blocks.reshape(P * PAGE, D)[:n].contiguous().view(torch.float8_e4m3fn).double() * g
    raw = blocks.reshape(P * 2, BLOCK // 2)
    code = raw[:, : HALF * 64].reshape(-1, 64)[:n].long()
    sc = raw[:, HALF * 64:].reshape(-1, 8)[:n].contiguous().view(torch.float8_e4m3fn).double()
    mag = _grid(2, 1, 1, 6.0)
    val = torch.stack([code % 16, code // 16], -1).reshape(n, D)
    val = torch.where(val >= 8, -mag[val % 8], mag[val % 8])
    return (val.reshape(n, 8, 16) * sc[..., None]).reshape(n, D) * g


def _exact_attend(st, q, lengths, dtype):
    c = st["c"]
    S, hkv, G = c["streams"], c["hkv"], c["hq"] // c["hkv"]
    R = q.shape[0] // S
    out = torch.empty(S * R, c["hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.empty(S * R, c["hq"], dtype=torch.float64, device="cuda")
    for i in range(S):
        n = lengths[i]
        for h in range(hkv):
            K, V = _exact_head(st, "k", i, h, n, dtype), _exact_head(st, "v", i, h, n, dtype)
            if "k_rows" in st:
                at = st["row_pos"][i * R: (i + 1) * R]
                for w, X in (("k", K), ("v", V)):
                    X[torch.from_numpy(at).cuda().long()] = _exact_quantised(st[w + "_rows"][i * R: (i + 1) * R, h].double(),
                                                                             st[w + "_scale"][h].double().expand(R))
            back = torch.from_numpy(st["row_pos"][i * R: (i + 1) * R].astype(np.int64)).cuda()[:, None] - torch.arange(n, device="cuda")[None]
            see = back >= 0
            if "anc" in st:
                see &= (back > 63) | (((st["anc"][i * R: (i + 1) * R, None] >> back.clamp(0, 63)) & 1) == 1)
            for e in range(h * G, (h + 1) * G):
                s = torch.where(see, q[i * R: (i + 1) * R, e].double() @ K.T * SCALE, -math.inf)
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                z = p.sum(-1, keepdim=True)
                out[i * R: (i + 1) * R, e] = p @ V / z
                lse[i * R: (i + 1) * R, e] = (m + z.log())[:, 0]
    return out, lse


def _exact_evicted(st):
    """Mass and positions after the eviction, and for each (stream, head) the slots that fill the first
    keep[s] slots."""
    c = st["c"]
    mass, pos = st["mass0"].cpu().numpy().astype(np.float64), st["pos0"].cpu().numpy().astype(np.int64)
    src = {}
    for i, (L, n) in enumerate(zip(st["lengths"], st["keep"])):
        for h in range(c["hkv"]):
            m, p = mass[i, h, :L], pos[i, h, :L]
            guard = (p < SINK) | (p >= st["next_pos"][i] - c["recent"])
            first = np.lexsort((np.arange(L), -m, ~guard))[:n]
            stays = np.zeros(L, bool)
            stays[first] = True
            take = np.arange(n)
            take[~stays[:n]] = np.flatnonzero(stays[n:]) + n
            src[i, h] = take
            mass[i, h, :L], pos[i, h, :L] = np.concatenate([m[take], np.zeros(L - n)]), np.concatenate([p[take], np.full(L - n, -1)])
    return mass, pos, src


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["kind"] == "store":
        out = []
        for w in ("k", "v"):
            x = st[w + "_rows"].double()
            if w == "k" and c["rope"]:
                t = torch.from_numpy(st["row_pos"].astype(np.int64)).cuda()
                co, si = st["cos"][t].double()[:, None], st["sin"][t].double()[:, None]
                x = torch.cat([x[..., :64] * co - x[..., 64:] * si, x[..., 64:] * co + x[..., :64] * si], -1)
            out.append(_exact_quantised(x, st[w + "_scale"].double().view(1, -1).expand(x.shape[:2])))
        return out
    if c["kind"] == "attend":
        return list(_exact_attend(st, st["q"], st["lengths"], "fp4"))
    if c["kind"] == "mass":
        S, hkv, G, R = c["streams"], c["hkv"], c["hq"] // c["hkv"], c["rows"]
        mass = st["mass"].double()
        for i, n in enumerate(st["lengths"]):
            see = torch.from_numpy(st["row_pos"][i * R: (i + 1) * R].astype(np.int64)).cuda()[:, None] >= torch.arange(n, device="cuda")[None]
            for h in range(hkv):
                K = _exact_head(st, "k", i, h, n, c["dtype"])
                add = torch.zeros(n, dtype=torch.float64, device="cuda")
                for e in range(h * G, (h + 1) * G):
                    w = torch.exp(st["q"][i * R: (i + 1) * R, e].double() @ K.T * SCALE - st["lse"][i * R: (i + 1) * R, e, None].double())
                    add += torch.where(see, w, 0.0).sum(0)
                mass[i, h, :n] = (mass[i, h, :n] * c["decay"] if c["decay"] else 0.0) + add
        return mass
    mass, pos, src = _exact_evicted(st)
    fine = {"mass": torch.from_numpy(mass), "pos": torch.from_numpy(pos).int()}
    for w in ("k", "v"):
        for (i, h), take in src.items():
            f = torch.from_numpy(take).cuda()
            d = torch.arange(len(take), device="cuda")
            f, d = f[f != d], d[f != d]
            if c["dtype"] == "fp4":
                for a, b in ((0, 64), (HALF * 64, 8)):
                    flat = st[w + "_pool"].view(-1)
                    at = lambda j: ((st["table"][i, j // PAGE].long() * c["hkv"] + h) * BLOCK + (j // HALF % 2) * (BLOCK // 2) + a + j % HALF * b)[:, None] + torch.arange(b, device="cuda")  # noqa: E731, E501
                    flat[at(d)] = flat[at(f)]
            else:
                rows = st[w + "_pool"].view(torch.uint8 if c["dtype"] == "fp8" else torch.bfloat16).view(-1, D)
                at = lambda j: (st["table"][i, j // PAGE].long() * c["hkv"] + h) * PAGE + j % PAGE  # noqa: E731
                rows[at(d)] = rows[at(f)]
    if c["dtype"] == "fp4":
        fine["out"], fine["lse"] = _exact_attend(st, st["q"], [int(n) for n in st["keep"]], "fp4")
        return fine
    return dict(fine, k=st["k_pool"].double(), v=st["v_pool"].double())
