"""Block bounds, block selection and attention over selected blocks on the GPU, each against its definition in 64
bits; the whole step as it is used."""

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests.gpu64 import SCALE, U, LongCase, assert_within, last_rows

pytestmark = pytest.mark.gpu

KVS = ["bf16", "fp8", "fp4"]


def plain_values(c, s, w, g):
    """K or V of a stream and head without the head's scale, float64 [L][128]."""
    x = c.values(s, w, g)
    return x if c.kv == "bf16" else x / (c.v_scale if w else c.k_scale)[g].double()


def bound_store(c, block, fill=3.0):
    """Bounds of a case's pool and slabs, filled with a value that no block has."""
    per = 256 // block
    b = B.make_bounds(c.num_pages, c.hkv, block)
    b.pool.fill_(fill)
    slabs = [None] * len(c.lengths)
    for s, (k, _) in c.slabs.items():
        slabs[s] = torch.full((c.hkv, k.shape[1] * per, 2, 128), fill, dtype=torch.bfloat16, device="cuda")
    b.slabs = slabs if c.slabs else None
    return b


def bound_view(c, b, s, blk):
    """[hkv][2][128] of one block, as a view."""
    if s in c.slabs:
        return b.slabs[s][:, blk]
    per = 256 // b.block
    return b.pool[int(c.segs[s].page_table[blk // per]), :, blk % per]


def exact_bounds(c, s, blk, block):
    out = torch.empty(c.hkv, 2, 128, dtype=torch.float64, device="cuda")
    for g in range(c.hkv):
        x = plain_values(c, s, 0, g)[blk * block: (blk + 1) * block].nan_to_num(nan=0.0, posinf=float("inf"), neginf=float("-inf"))
        out[g, 0], out[g, 1] = x.amin(0), x.amax(0)
    return out


# ---------------------------------------------------------------- bounds
@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("block", [64, 128, 256])
def test_bounds(kv, block):
    lengths = [1, 63, 64, 65, 700, 1025]
    c = LongCase(kv, lengths, [True, True, False, True, False, True], 8, 2, 11)
    b = bound_store(c, block)
    rs = np.concatenate([np.full(L, s) for s, L in enumerate(lengths)])
    rp = np.concatenate([np.arange(L) for L in lengths])
    B.tfpa_key_bounds(c.cache, c.segs, b, rs, rp)
    for s, L in enumerate(lengths):
        n = -(-L // block)
        for blk in range(n):
            assert torch.allclose(bound_view(c, b, s, blk).double(), exact_bounds(c, s, blk, block), rtol=1e-7, atol=0), (s, blk)
        last = 256 // block * -(-L // 256)
        assert all((bound_view(c, b, s, blk) == 3.0).all() for blk in range(n, last))
    assert int(c.err.item()) == 0


def test_only_the_blocks_of_the_rows_are_taken():
    c = LongCase("bf16", [1000, 600], [True, False], 8, 2, 12)
    b = bound_store(c, 64)
    B.tfpa_key_bounds(c.cache, c.segs, b, [0, 0, 1, 0, 0], [127, 128, 599, 500, 127])      # overlapping runs too
    for s, want in ((0, {1, 2, 7}), (1, {9})):
        for blk in range(-(-c.lengths[s] // 64)):
            got = bound_view(c, b, s, blk)
            if blk in want:
                assert torch.equal(got.double(), exact_bounds(c, s, blk, 64))
            else:
                assert (got == 3.0).all(), (s, blk)


def test_bounds_of_overwritten_rows_shrink():
    c = LongCase("bf16", [130], [True], 8, 2, 13)
    b = bound_store(c, 64)
    big = torch.full((1, 2, 128), 50.0, dtype=torch.bfloat16, device="cuda")
    B.tfpa_write_kv(c.cache, c.segs, big, big, [0], [129])
    B.tfpa_key_bounds(c.cache, c.segs, b, [0], [129])
    assert (bound_view(c, b, 0, 2)[:, 1] == 50).all()
    B.tfpa_write_kv(c.cache, c.segs, -big / 10, big, [0], [129])
    B.tfpa_key_bounds(c.cache, c.segs, b, [0], [129])
    assert torch.equal(bound_view(c, b, 0, 2).double(), exact_bounds(c, 0, 2, 64)) and (bound_view(c, b, 0, 2)[:, 1] < 50).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_bounds_of_keys_that_are_no_numbers(kv):
    c = LongCase(kv, [256], [True], 8, 2, 14)
    page = c._page(0, 0, 0)
    if kv == "bf16":
        page[:, 0, 5], page[:, 70, 6], page[:, 71, 6], page[:, 130:192, 7] = float("nan"), float("inf"), float("-inf"), float("nan")
        page[0, 192:256] = float("nan")
    else:
        page[:, 0, 5], page[:, 130:192, 7] = 0x7F, 0xFF
        page[0, 192:256] = 0xFF
    b = bound_store(c, 64)
    B.tfpa_key_bounds(c.cache, c.segs, b, np.zeros(256), np.arange(256))
    for blk in range(4):
        assert torch.allclose(bound_view(c, b, 0, blk).double(), exact_bounds(c, 0, blk, 64), rtol=1e-7, atol=0)
    assert (bound_view(c, b, 0, 3)[0] == 0).all()


def test_bounds_on_a_page_out_of_range():
    c = LongCase("fp8", [700], [True], 8, 2, 15)
    b = bound_store(c, 128)
    good = c.segs[0].page_table.clone()
    for bad in (-1, c.num_pages):
        c.segs[0].page_table[1] = bad
        B.tfpa_key_bounds(c.cache, c.segs, b, np.zeros(700), np.arange(700))
        c.segs[0].page_table.copy_(good)
        assert int(c.err.item()) == 1
        assert [bool((bound_view(c, b, 0, i) == 3.0).all()) for i in range(6)] == [False, False, True, True, False, False]


# ---------------------------------------------------------------- selection
def scores(c, b, q, r, s, n, g):
    """Of every head sum and block, float64 [n]: the definition, term by term."""
    G = c.hq // c.hkv
    e = torch.stack([bound_view(c, b, s, i)[g] for i in range(n)]).double()
    x = q[r, g * G: (g + 1) * G].double()
    up, down = torch.where(x < 0, 0.0, x).sum(0), torch.where(x > 0, 0.0, x).sum(0)
    return (up * e[:, 1]).sum(-1) + (down * e[:, 0]).sum(-1)


def choose(score, last, nsel, sink, recent, absent=()):
    b = np.array([i for i in range(last + 1) if i not in absent])
    sc = np.where(np.isnan(score), np.inf, score)[b]
    nan = np.isnan(score)[b]
    forced = (b < sink) | (b > last - recent)
    got = np.sort(b[np.lexsort((b, -sc, ~nan, ~forced))[:nsel]])
    return np.concatenate([got, np.full(nsel - len(got), -1)]).astype(np.int32)


def random_bounds(c, block, seed, like=None):
    b = bound_store(c, block)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    for t in [b.pool] + [x for x in (b.slabs or []) if x is not None]:
        mid = torch.randn(*t.shape[:-2], 1, 128, generator=g, device="cuda")
        half = torch.rand(*t.shape[:-2], 1, 128, generator=g, device="cuda") * 2
        t.copy_(torch.cat([mid - half, mid + half], -2))
    return b


def check_choice(c, b, q, rs, rp, nsel, sink, recent, got=None, absent=()):
    if got is None:
        got = torch.full((len(rs) + 2, c.hkv, nsel), 77, dtype=torch.int32, device="cuda")
        B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, got[1:-1], sink=sink, recent=recent)
        assert (got[[0, -1]] == 77).all()
        got = got[1:-1]
    a = got.cpu().numpy()
    for r, (s, p) in enumerate(zip(rs, rp)):
        for g in range(c.hkv):
            last = int(p) // b.block
            want = choose(scores(c, b, q, r, int(s), last + 1, g).cpu().numpy(), last, nsel, sink, recent, absent)
            assert np.array_equal(a[r, g], want), (r, g, a[r, g], want)


@pytest.mark.parametrize("block", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,nsel,sink,recent", [(8, 2, 16, 1, 2), (6, 1, 1, 0, 0), (5, 5, 7, 0, 1), (20, 1, 64, 3, 0), (32, 2, 200, 0, 0), (8, 8, 12, 4, 8)])
def test_selection(block, hq, hkv, nsel, sink, recent):
    lengths = [1, 64, 65, 5000, 20001, 4097]
    c = LongCase("bf16", lengths, [True, False, True, True, True, False], hq, hkv, 21)
    b = random_bounds(c, block, 22)
    rs, rp = last_rows(lengths, [1, 1, 2, 3, 1, 1])
    rs, rp = np.append(rs, [4, 3]), np.append(rp, [0, 2500])            # rows in the middle of a stream
    check_choice(c, b, c.q(len(rs)), rs, rp, nsel, sink, recent)
    assert int(c.err.item()) == 0


def one(L=20000, hq=4, hkv=1, seed=31):
    c = LongCase("bf16", [L], [True], hq, hkv, seed)
    return c, random_bounds(c, 64, seed + 1), [0], [L - 1]


def blocks_of(c, b, s=0):
    per = 256 // b.block
    n = -(-c.lengths[s] // b.block)
    return [(int(c.segs[s].page_table[i // per]), i % per) for i in range(n)]


@pytest.mark.parametrize("nsel", [1, 2, 63, 64, 100, 312])
def test_all_blocks_alike(nsel):
    """Ties go to the lower block, however many they are."""
    c, b, rs, rp = one()
    b.pool[:] = b.pool[0, 0, 0]
    check_choice(c, b, c.q(1), rs, rp, nsel, 0, 1)
    b.pool.zero_()
    check_choice(c, b, c.q(1), rs, rp, nsel, 0, 0)


@pytest.mark.parametrize("copies", [2, 30, 150])
def test_ties_at_the_border(copies):
    c, b, rs, rp = one()
    q = c.q(1)
    at = blocks_of(c, b)
    order = np.argsort(-scores(c, b, q, 0, 0, len(at), 0).cpu().numpy())
    src = at[order[20]]
    for i in np.random.default_rng(3).permutation(len(at))[:copies]:
        b.pool[at[i][0], :, at[i][1]] = b.pool[src[0], :, src[1]]
    for nsel in (15, 21, 25, 40):
        check_choice(c, b, q, rs, rp, nsel, 0, 0)


def test_scores_nearer_than_float32_can_tell():
    """Blocks whose scores differ by far less than a float32 step: one small dim under many large ones."""
    c, b, rs, rp = one(hq=4)
    q = c.q(1)
    q[..., 127] = 2.0 ** -18
    base = b.pool[0, 0, 0].clone()
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    b.pool[:] = base
    b.pool[..., 1, 127] = torch.rand(b.pool.shape[:-2], generator=g, device="cuda").to(torch.bfloat16)
    b.pool[..., 0, 127] = -1.0
    for nsel in (1, 10, 50, 100, 200):
        check_choice(c, b, q, rs, rp, nsel, 0, 1)


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_scores_at_the_ends_of_float32(scale):
    """Products that overflow float32 (but not the choice) and ones that are next to nothing."""
    c, b, rs, rp = one()
    b.pool.mul_(scale)
    q = (c.q(1).float() * (1e9 if scale > 1 else 1e-9)).to(torch.bfloat16)
    check_choice(c, b, q, rs, rp, 20, 0, 1)


def test_bounds_that_are_no_numbers_or_infinite():
    c, b, rs, rp = one()
    at = blocks_of(c, b)
    q = c.q(1)
    q[0, :, 4] = 0.0
    for i, (d, w, v) in enumerate([(3, 0, float("nan")), (4, 1, float("inf")), (5, 1, float("inf")), (6, 0, float("-inf")), (7, 1, float("-inf"))]):
        p, j = at[40 + 7 * i]
        b.pool[p, :, j, w, d] = v
    for nsel in (1, 2, 3, 5, 30):
        check_choice(c, b, q, rs, rp, nsel, 0, 0)
    q[0, 1, 9] = float("nan")                          # every score is none: the first blocks
    check_choice(c, b, q, rs, rp, 9, 0, 2)
    q[0, 1, 9] = float("inf")
    check_choice(c, b, q, rs, rp, 9, 0, 2)


def test_blocks_on_a_page_out_of_range_are_not_chosen():
    c = LongCase("bf16", [3000], [True], 8, 2, 41)
    b = random_bounds(c, 64, 42)
    table = c.segs[0].page_table
    q = c.q(1)
    for bad in (-5, c.num_pages):
        keep = [int(table[0]), int(table[5])]
        want = {g: scores(c, b, q, 0, 0, 47, g).cpu().numpy() for g in range(2)}
        table[0], table[5] = bad, bad
        got = torch.zeros(1, 2, 47, dtype=torch.int32, device="cuda")
        small = torch.zeros(1, 2, 10, dtype=torch.int32, device="cuda")
        B.tfpa_select_blocks(c.cache, c.segs, b, q, [0], [2999], got, sink=2, recent=2)
        B.tfpa_select_blocks(c.cache, c.segs, b, q, [0], [2999], small, sink=2, recent=2)
        table[0], table[5] = keep[0], keep[1]
        assert int(c.err.item()) == 1
        absent = [0, 1, 2, 3, 20, 21, 22, 23]
        for g in range(2):
            for t, n in ((got, 47), (small, 10)):
                assert np.array_equal(t[0, g].cpu().numpy(), choose(want[g], 46, n, 2, 2, absent))


@pytest.mark.parametrize("L", [131072, 18432 * 64 - 5])
def test_selection_over_very_long_streams(L):
    """Pages that are named many times: the longest rows that a call takes, without their memory."""
    c = LongCase("bf16", [4096], [True], 8, 2, 51)
    b = random_bounds(c, 64, 52)
    n = -(-L // 256)
    table = torch.randint(0, c.num_pages, (n,), dtype=torch.int32, device="cuda")
    c.lengths, c.segs = [L], [B.Seg(L, page_table=table)]
    q, rs, rp = c.q(2), [0, 0], [L - 1, L // 2]
    got = torch.zeros(2, 2, 48, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, got, sink=1, recent=2)
    for r in range(2):
        for g in range(2):
            G = 4
            e = b.pool[table.long(), g].flatten(0, 1).double()
            x = q[r, g * G: (g + 1) * G].double()
            up, down = torch.where(x < 0, 0.0, x).sum(0), torch.where(x > 0, 0.0, x).sum(0)
            sc = ((up * e[:, 1]).sum(-1) + (down * e[:, 0]).sum(-1)).cpu().numpy()
            assert np.array_equal(got[r, g].cpu().numpy(), choose(sc[: rp[r] // 64 + 1], rp[r] // 64, 48, 1, 2))


# ---------------------------------------------------------------- attention
def attend64(c, q, rs, rp, lists, block):
    """out, lse and what each may be off by: as gpu64.attend has them, over the listed keys."""
    rows, G = len(rs), c.hq // c.hkv
    out, tol = (torch.zeros(rows, c.hq, 128, dtype=torch.float64, device="cuda") for _ in range(2))
    lse, ltol = (torch.zeros(rows, c.hq, dtype=torch.float64, device="cuda") for _ in range(2))
    a = lists.cpu().numpy()
    for s in sorted(set(int(x) for x in rs)):
        for g in range(c.hkv):
            K, V = c.values(s, 0, g), c.values(s, 1, g)
            for r in [r for r in range(rows) if rs[r] == s]:
                blk = a[r, g][a[r, g] >= 0].astype(np.int64)
                key = (blk[:, None] * block + np.arange(block)).reshape(-1)
                key = torch.from_numpy(key[key <= rp[r]]).cuda()
                h = slice(g * G, (g + 1) * G)
                if not len(key):
                    lse[r, h] = -torch.inf
                    continue
                Q, k, v = q[r, h].double(), K[key], V[key]
                x = SCALE * (Q @ k.T)
                xa = (SCALE * (Q.abs() @ k.abs().T)).amax(-1, keepdim=True)
                m = x.amax(-1, keepdim=True)
                e = (x - m).exp()
                z = e.sum(-1, keepdim=True)
                es = 2 * 128 * U * xa + 2.0 ** -20
                out[r, h], lse[r, h] = e @ v / z, (m + z.log())[:, 0]
                # over bf16 a weight is its first 8 bits and the rest, 2^-7 of it at most, rounded to 8 (2^-8 of that); else
                # it rounds to f16 (11 bits: 2^-11), below 2^-14 to a multiple of 2^-24
                wr = 2.0 ** -15 if c.kv == "bf16" else 2.0 ** -11
                tol[r, h] = (2.0 ** -8 * out[r, h].abs() + (e @ v.abs() / z) * (wr + 2 * es)
                             + len(key) * 2.0 ** -25 / z * v.abs().max() + 1e-30)
                ltol[r, h] = es[:, 0] + 4 * U * (lse[r, h].abs() + m[:, 0].abs() + 20)
    return out, lse, tol, ltol


def run_attend(c, q, rs, rp, lists, block, **kw):
    rows = len(rs)
    out = torch.full((rows + 2, c.hq, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((rows + 2, c.hq), 5.0, device="cuda")
    B.tfpa_decode_blocks(c.cache, c.segs, q, rs, rp, lists, block, SCALE, out[1:-1], lse[1:-1], **kw)
    torch.cuda.synchronize()
    assert (out[[0, -1]] == 5).all() and (lse[[0, -1]] == 5).all()
    return out[1:-1], lse[1:-1]


def check_attend(c, q, rs, rp, lists, block):
    out, lse = run_attend(c, q, rs, rp, lists, block)
    ref, rl, tol, ltol = attend64(c, q, rs, rp, lists, block)
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse), none) and (lse[none] < 0).all() and (out[none] == 0).all()
    assert_within(out, ref, tol, "out")
    assert_within(lse[~none], rl[~none], ltol[~none], "lse")
    return out, lse


def random_lists(c, rs, rp, nsel, block, seed, shuffle=False):
    rng = np.random.default_rng(seed)
    a = np.full((len(rs), c.hkv, nsel), -1, np.int32)
    for r, p in enumerate(rp):
        for g in range(c.hkv):
            n = int(p) // block + 1
            pick = np.append(rng.permutation(n - 1)[: nsel - 1], n - 1)
            pick = rng.permutation(pick) if shuffle else np.sort(pick)
            a[r, g, : len(pick)] = pick
            if shuffle:
                a[r, g] = rng.permutation(a[r, g])
    return torch.from_numpy(a).cuda()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("block", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,nsel", [(8, 2, 16), (6, 1, 1), (5, 5, 3), (20, 1, 9), (32, 2, 33), (40, 1, 5)])
def test_attention(kv, block, hq, hkv, nsel):
    lengths = [1, 64, 65, 700, 4097, 5000]
    c = LongCase(kv, lengths, [True, False, True, False, True, True], hq, hkv, 61)
    rs, rp = last_rows(lengths, [1, 1, 2, 3, 1, 2])
    rs, rp = np.append(rs, [5, 4]), np.append(rp, [0, 2500])
    check_attend(c, c.q(len(rs)), rs, rp, random_lists(c, rs, rp, nsel, block, 62, shuffle=nsel in (9, 33)), block)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("kv", KVS)
def test_lists_with_odd_entries(kv):
    """Empty lists, entries behind the row, far numbers, one block twice."""
    c = LongCase(kv, [5000, 300], [True, False], 8, 2, 63)
    rs, rp = [0, 0, 0, 0, 1, 1], [4999, 4998, 70, 4000, 299, 0]
    a = torch.full((6, 2, 6), -1, dtype=torch.int32, device="cuda")
    big = 2**31 - 1
    a[1] = torch.tensor([[-1, 78, -7, -2**31, 3, -1], [big, 79, 2**25, 77, 0, 2**24 + 1]])
    a[2] = torch.tensor([[1, 2, 3, 78, -1, -1], [2, 3, 4, 5, 6, 7]])      # the second list has nothing that the row sees
    a[3] = torch.tensor([[5, 5, 5, 9, 62, 62], [62, -1, 62, 0, 0, 63]])
    a[4] = torch.tensor([[4, 0, 1, 2, 3, 5], [4, 4, -1, -1, -1, -1]])
    a[5] = torch.tensor([[0, 1, -1, -1, -1, -1], [-1, -1, -1, -1, -1, 0]])
    check_attend(c, c.q(6), rs, rp, a, 64)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("kv", KVS)
def test_what_lies_behind_a_row_does_not_reach_it(kv):
    """Keys after the row's position, in its own block: not numbers, in K and V."""
    c = LongCase(kv, [1000], [True], 8, 2, 64)
    rs, rp = [0, 0], [900, 897]
    lists = random_lists(c, rs, rp, 4, 64, 65)
    q = c.q(2)
    want = run_attend(c, q, rs, rp, lists, 64)
    for w in (0, 1):
        c._spoil(0, w, 3, 901 - 768)
    got = run_attend(c, q, rs, rp, lists, 64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_infinite_and_nan_keys_that_are_seen():
    c = LongCase("bf16", [300], [True], 4, 2, 66)
    page = c._page(0, 0, 0)
    page[0, 10, 3] = float("nan")
    c._page(0, 1, 0)[1, 20, 5] = float("inf")
    lists = torch.zeros(1, 2, 2, dtype=torch.int32, device="cuda")
    lists[..., 1] = 4
    out, lse = run_attend(c, c.q(1), [0], [299], lists, 64)
    assert torch.isnan(out[0, :2]).all() and torch.isnan(lse[0, :2]).all()
    assert torch.isfinite(lse[0, 2:]).all() and (out[0, 2:, 5] == torch.inf).all() and torch.isfinite(out[0, 2:, 6]).all()


@pytest.mark.parametrize("kv", KVS)
def test_attention_on_a_page_out_of_range(kv):
    c = LongCase(kv, [2000], [True], 8, 2, 67)
    q, rs, rp = c.q(1), [0], [1999]
    lists = torch.tensor([0, 5, 9, 20, 31], dtype=torch.int32, device="cuda").expand(1, 2, 5).contiguous()
    less = torch.tensor([0, -1, 9, -1, 31], dtype=torch.int32, device="cuda").expand(1, 2, 5).contiguous()
    want = check_attend(c, q, rs, rp, less, 64)
    keep = c.segs[0].page_table.clone()
    for bad in (-1, c.num_pages):
        c.segs[0].page_table[1], c.segs[0].page_table[5] = bad, bad
        got = run_attend(c, q, rs, rp, lists, 64)
        c.segs[0].page_table.copy_(keep)
        assert int(c.err.item()) == 1
        c.err.zero_()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_large_scores():
    """Scores of some thousands, whose exponentials would overflow; one key takes all."""
    c = LongCase("bf16", [3000], [True], 8, 2, 68)
    check_attend(c, c.q(1, scale=200.0), [0], [2999], random_lists(c, [0], [2999], 20, 64, 69), 64)


@pytest.mark.parametrize("kv", KVS)
def test_a_row_is_the_same_bytes_alone_and_in_a_batch(kv):
    """Batched or alone, paged or in a slab, from another host thread's stream: one arithmetic."""
    lengths = [3000] * 70 + [700, 9000]
    c = LongCase(kv, lengths, [True] * 35 + [False] * 10 + [True] * 27, 8, 2, 70)
    rs, rp = last_rows(lengths, [1] * 70 + [3, 2])
    lists = random_lists(c, rs, rp, 12, 64, 71)
    q = c.q(len(rs))
    out, lse = run_attend(c, q, rs, rp, lists, 64)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for r in (0, 5, 40, 69, 71, len(rs) - 1):
        o, l = run_attend(c, q[r:r + 1].contiguous(), rs[r:r + 1], rp[r:r + 1], lists[r:r + 1].contiguous(), 64, stream=s)
        assert torch.equal(o[0], out[r]) and torch.equal(l[0], lse[r])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kv", KVS)
def test_a_step_of_long_streams(kv):
    """Projection rows -> cache -> bounds -> blocks -> attention, three steps; the blocks are those of the exact scores and
    the output is the attention over them.  With room for every block it is tfpa_decode's."""
    lengths = [2000, 700, 5003]
    c = LongCase(kv, lengths, [True, False, True], 8, 2, 81)
    b = bound_store(c, 64)
    rs = np.concatenate([np.full(L, s) for s, L in enumerate(lengths)])
    B.tfpa_key_bounds(c.cache, c.segs, b, rs, np.concatenate([np.arange(L) for L in lengths]))
    cos, sin = (torch.empty(6000, 64, device="cuda") for _ in range(2))
    B.tfpa_rope_table(B.RopeSpec(1e4, scaling="ramp", factor=4.0, orig_len=2048, low=1.0, high=32.0), 0, cos, sin)
    w = torch.ones(128, device="cuda")
    tab = B.SegTable(c.segs)
    for step in range(3):
        x = torch.randn(6, 12, 128, generator=c.g, device="cuda").to(torch.bfloat16)
        rs, rp = last_rows(c.lengths, [2, 2, 2])
        q = torch.empty(6, 8, 128, dtype=torch.bfloat16, device="cuda")
        lists, full = (torch.empty(6, 2, n, dtype=torch.int32, device="cuda") for n in (10, 80))
        out, lse = torch.empty_like(q), torch.empty(6, 8, device="cuda")
        B.tfpa_write_qkv(c.cache, tab, x[:, :8], x[:, 8:10], x[:, 10:], q, rs, rp, q_weight=w, k_weight=w, rope_cos=cos, rope_sin=sin)
        B.tfpa_key_bounds(c.cache, tab, b, rs, rp)
        B.tfpa_select_blocks(c.cache, tab, b, q, rs, rp, lists, sink=1, recent=2)
        B.tfpa_decode_blocks(c.cache, tab, q, rs, rp, lists, 64, SCALE, out, lse)
        check_choice(c, b, q, rs, rp, 10, 1, 2, got=lists)
        o, l = check_attend(c, q, rs, rp, lists, 64)
        assert torch.equal(o, out) and torch.equal(l, lse)
        B.tfpa_select_blocks(c.cache, tab, b, q, rs, rp, full, sink=1, recent=2)
        o, l = check_attend(c, q, rs, rp, full, 64)
        dense, dl = torch.empty_like(q), torch.empty_like(lse)
        B.tfpa_decode(c.cache, tab, q, rs, rp, SCALE, B.make_scratch(16, 8), dense, dl)
        _, _, tol, ltol = attend64(c, q, rs, rp, full, 64)
        assert ((o.double() - dense.double()).abs() <= 2 * tol).all() and ((l - dl).abs().double() <= 2 * ltol).all()
    assert int(c.err.item()) == 0


def test_a_step_captured_and_replayed():
    """The four calls in one graph, replayed with other rows; an eager step on another stream's cache in between."""
    c = LongCase("fp8", [3000, 1500], [True, False], 8, 2, 82)
    b = bound_store(c, 128)
    rs, rp = last_rows(c.lengths, [1, 1])
    every = np.concatenate([np.full(L, s) for s, L in enumerate(c.lengths)]), np.concatenate([np.arange(L) for L in c.lengths])
    B.tfpa_key_bounds(c.cache, c.segs, b, *every)
    cos, sin = (torch.rand(3100, 64, device="cuda") for _ in range(2))
    x = torch.randn(2, 12, 128, generator=c.g, device="cuda").to(torch.bfloat16)
    q, out = (torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lists = torch.empty(2, 2, 6, dtype=torch.int32, device="cuda")

    def step():
        B.tfpa_write_qkv(c.cache, c.segs, x[:, :8], x[:, 8:10], x[:, 10:], q, rs, rp, rope_cos=cos, rope_sin=sin)
        B.tfpa_key_bounds(c.cache, c.segs, b, rs, rp)
        B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, sink=0, recent=1)
        B.tfpa_decode_blocks(c.cache, c.segs, q, rs, rp, lists, 128, SCALE, out)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step()
    for _ in range(2):
        x.copy_(torch.randn(2, 12, 128, generator=c.g, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (q, lists, out, b.pool)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, (q, lists, out, b.pool)))
        check_choice(c, b, q, rs, rp, 6, 0, 1, got=lists)


def test_calls_of_several_threads_at_once():
    import threading
    cases = []
    for i in range(4):
        c = LongCase(KVS[i % 3], [2500 + 100 * i, 800], [True, False], 8, 2, 90 + i)
        b = random_bounds(c, 64, 95 + i)
        rs, rp = last_rows(c.lengths, [2, 1])
        cases.append((c, b, c.q(3), rs, rp))
    torch.cuda.synchronize()
    got, wrong = [None] * 4, []

    def work(i):
        try:
            c, b, q, rs, rp = cases[i]
            s = torch.cuda.Stream()
            for _ in range(20):
                lists = torch.empty(3, 2, 8, dtype=torch.int32, device="cuda")
                out, lse = torch.empty_like(q), torch.empty(3, 8, device="cuda")
                s.wait_stream(torch.cuda.current_stream())
                B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, stream=s)
                B.tfpa_decode_blocks(c.cache, c.segs, q, rs, rp, lists, 64, SCALE, out, lse, stream=s)
                s.synchronize()
                if got[i] is not None and not all(torch.equal(u, v) for u, v in zip(got[i], (lists, out, lse))):
                    wrong.append(i)
                got[i] = (lists, out, lse)
        except Exception as e:                          # noqa: BLE001
            wrong.append(repr(e))

    t = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [x.start() for x in t]
    [x.join() for x in t]
    assert not wrong
    for (c, b, q, rs, rp), (lists, out, lse) in zip(cases, got):
        check_choice(c, b, q, rs, rp, 8, 0, 1, got=lists)
        o, l = check_attend(c, q, rs, rp, lists, 64)
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("hq,hkv,rows", [(8, 2, 1), (32, 2, 2), (8, 2, 90)])
def test_long_lists(kv, hq, hkv, rows):
    """Dozens of key stages a part, so that every buffer is filled again and again; rows enough that a CTA takes several
    parts of a list."""
    c = LongCase(kv, [30000, 9000], [True, False], hq, hkv, 72)
    rs, rp = last_rows(c.lengths, [rows, rows])
    nsel = 300 if rows < 10 else 60
    check_attend(c, c.q(len(rs)), rs, rp, random_lists(c, rs, rp, nsel, 64, 73), 64)
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (32, 2), (6, 1)])
def test_a_row_is_the_same_bytes_whatever_parts_a_cta_takes(kv, hq, hkv):
    """Batches of 1 to 600 rows: one, two, four or eight parts of a list in a CTA, for lists of two to eight parts."""
    c = LongCase(kv, [4000, 2000], [True, False], hq, hkv, 74)
    rs, rp = last_rows(c.lengths, [300, 300])
    q = c.q(600)
    for nsel in (3, 11, 40):
        lists = random_lists(c, rs, rp, nsel, 64, 75)
        out, lse = run_attend(c, q, rs, rp, lists, 64)
        for n in (1, 25, 50, 120, 250):
            o, l = run_attend(c, q[:n].contiguous(), rs[:n], rp[:n], lists[:n].contiguous(), 64)
            assert torch.equal(o.view(torch.int16), out[:n].view(torch.int16)) and torch.equal(l, lse[:n]), (nsel, n)


@pytest.mark.parametrize("block", [64, 256])
def test_rows_of_a_run_share_their_reads(block):
    """Runs of 2, 3, 4, 5 and 9 rows that cross a block's border, in one call and row by row: the same blocks."""
    lengths = [4099, 4098, 4100, 8193, 4104]
    c = LongCase("bf16", lengths, [True, False, True, True, True], 8, 2, 76)
    b = random_bounds(c, block, 77)
    rs, rp = last_rows(lengths, [2, 3, 4, 5, 9])
    q = c.q(len(rs))
    got = torch.empty(len(rs), 2, 12, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, got, sink=1, recent=2)
    check_choice(c, b, q, rs, rp, 12, 1, 2, got=got)
    for r in range(len(rs)):
        one_row = torch.empty(1, 2, 12, dtype=torch.int32, device="cuda")
        B.tfpa_select_blocks(c.cache, c.segs, b, q[r:r + 1].contiguous(), rs[r:r + 1], rp[r:r + 1], one_row, sink=1, recent=2)
        assert torch.equal(one_row[0], got[r])


def test_a_prompt_chunk_over_its_own_blocks():
    """Hundreds of rows of one run, each with blocks of its own: bounds, choice and attention."""
    c = LongCase("fp8", [2500], [True], 8, 2, 78)
    b = bound_store(c, 64)
    B.tfpa_key_bounds(c.cache, c.segs, b, np.zeros(2500), np.arange(2500))
    rs, rp = np.zeros(700, np.int32), np.arange(1800, 2500, dtype=np.int32)
    q = c.q(700)
    lists = torch.empty(700, 2, 9, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, sink=1, recent=2)
    pick = np.arange(0, 700, 29)
    check_choice(c, b, q[torch.from_numpy(pick).cuda()].contiguous(), rs[pick], rp[pick], 9, 1, 2,
                 got=lists[torch.from_numpy(pick).cuda()])
    check_attend(c, q, rs, rp, lists, 64)


def test_after_an_eviction_the_bounds_are_taken_anew():
    """tfpa_evict_kv moves keys: with the bounds of all rows taken again, blocks and attention are those of the cut stream."""
    c = LongCase("bf16", [2000], [True], 8, 2, 79)
    b = bound_store(c, 64)
    cap = 2048
    mass = torch.rand(1, 2, cap, generator=c.g, device="cuda")
    moves = B.make_moves(1, 2, cap)
    B.tfpa_evict_kv(c.cache, c.segs, [900], mass, moves, sink=4, recent=64)
    c.lengths, c.segs = [900], [B.Seg(900, page_table=c.segs[0].page_table)]
    B.tfpa_key_bounds(c.cache, c.segs, b, np.zeros(900), np.arange(900))
    for blk in range(15):
        assert torch.equal(bound_view(c, b, 0, blk).double(), exact_bounds(c, 0, blk, 64))
    q, rs, rp = c.q(1), [0], [899]
    lists = torch.empty(1, 2, 5, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, sink=1, recent=1)
    check_choice(c, b, q, rs, rp, 5, 1, 1, got=lists)
    check_attend(c, q, rs, rp, lists, 64)


# ---------------------------------------------------------------- ends of what the calls allow
@pytest.mark.parametrize("kv", KVS)
def test_pages_far_into_a_pool(kv):
    """The same rows on a pool's first pages and on its last, whose elements lie past 2^32 bytes: the same bytes."""
    row = {"bf16": 256, "fp8": 128, "fp4": 72}[kv]
    hkv, hq, L = 2, 8, 1500
    n = 2**32 // (row * 256 * hkv) + 40
    pool = [torch.empty(n * hkv * 256 * row, dtype=torch.uint8, device="cuda") for _ in range(2)]
    one = torch.full((hkv,), 0.01, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = B.Cache(kv, hq, hkv, *pool, *((None, None) if kv == "bf16" else (one, one)), err, n)
    b = B.make_bounds(n, hkv, 64)
    gen = torch.Generator(device="cuda").manual_seed(91)
    x = torch.randn(L, hq + 2 * hkv, 128, generator=gen, device="cuda").to(torch.bfloat16)
    got = []
    for first in (3, n - 6):
        seg = B.Seg(L, page_table=torch.arange(first, first + 6, dtype=torch.int32, device="cuda"))
        rs, rp = np.zeros(L, np.int32), np.arange(L, dtype=np.int32)
        q, out = (torch.empty(L, hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lists = torch.empty(L, hkv, 5, dtype=torch.int32, device="cuda")
        B.tfpa_write_qkv(cache, [seg], x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q, rs, rp)
        B.tfpa_key_bounds(cache, [seg], b, rs, rp)
        B.tfpa_select_blocks(cache, [seg], b, q, rs, rp, lists, sink=1, recent=1)
        B.tfpa_decode_blocks(cache, [seg], q, rs, rp, lists, 64, SCALE, out)
        lo, hi = b.pool[first:first + 6].float().unbind(3)
        got.append([q, lists, out, b.pool[first:first + 6].clone()])
        assert (lo[:5] < 0).all() and (hi[:5] > 0).all() and torch.isfinite(out.float()).all()
    assert int(err.item()) == 0
    assert all(torch.equal(u, v) for u, v in zip(*got))
    k = x[L - 1, hq:hq + hkv].float()
    w = x[L - 1, hq + hkv:].float()
    kk, vv = (torch.empty(1, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    B.tfpa_read_kv(cache, [seg], kk, vv, [0], [L - 1])
    # a value is off by half a step of its type at most; bf16 stores it as it is, e2m1's largest step is 2 of 6
    off = {"bf16": 0.0, "fp8": 2.0 ** -4, "fp4": 0.0}[kv]
    for have, want in ((kk, k), (vv, w)):
        d = (have[0].float() - want).abs()
        if kv == "fp4":
            assert (d <= want.abs().view(hkv, 8, 16).amax(-1).repeat_interleave(16, -1) * (1 / 6 + 2.0 ** -4 + 2.0 ** -8)).all()
        else:
            assert (d <= off * want.abs() + 2.0 ** -10 * 0.01 * (off > 0) + 2.0 ** -8 * want.abs() * (off > 0)).all()


@pytest.mark.parametrize("kv", KVS)
def test_the_same_position_twice(kv):
    """Two rows of one call at one position: both have their q and attention, the position holds a K and V of theirs."""
    c = LongCase(kv, [700], [True], 8, 2, 92)
    x = torch.randn(2, 12, 128, generator=c.g, device="cuda").to(torch.bfloat16)
    x[1] = x[0]
    x[1, :8] = -x[0, :8]
    q = torch.empty(2, 8, 128, dtype=torch.bfloat16, device="cuda")
    rs, rp = [0, 0], [699, 699]
    B.tfpa_write_qkv(c.cache, c.segs, x[:, :8], x[:, 8:10], x[:, 10:], q, rs, rp)
    assert torch.equal(q, x[:, :8])
    b = bound_store(c, 64)
    every = np.zeros(700, np.int32), np.arange(700, dtype=np.int32)
    B.tfpa_key_bounds(c.cache, c.segs, b, np.concatenate([every[0]] * 2), np.concatenate([every[1]] * 2))
    for blk in range(11):
        assert torch.equal(bound_view(c, b, 0, blk).double(), exact_bounds(c, 0, blk, 64))
    lists = torch.empty(2, 2, 4, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, sink=0, recent=1)
    check_choice(c, b, q, rs, rp, 4, 0, 1, got=lists)
    check_attend(c, q, rs, rp, lists, 64)


@pytest.mark.parametrize("kv", KVS)
def test_a_very_long_list_of_few_blocks(kv):
    """A list of 2^20 entries, all but the first, a middle one and the last of them empty."""
    c = LongCase(kv, [5000], [True], 4, 1, 93)
    lists = torch.full((1, 1, 2**20), -1, dtype=torch.int32, device="cuda")
    lists[0, 0, 0], lists[0, 0, 2**19 + 77], lists[0, 0, -1] = 5, 78, 0
    check_attend(c, c.q(1), [0], [4999], lists, 64)
    assert int(c.err.item()) == 0


def test_many_query_heads_of_one_kv_head():
    """128 query heads of one kv head, in the selection and in the attention."""
    c = LongCase("bf16", [3000, 200], [True, False], 128, 1, 94)
    b = random_bounds(c, 64, 95)
    rs, rp = last_rows(c.lengths, [3, 1])
    q = c.q(len(rs))
    lists = torch.empty(len(rs), 1, 9, dtype=torch.int32, device="cuda")
    B.tfpa_select_blocks(c.cache, c.segs, b, q, rs, rp, lists, sink=1, recent=2)
    check_choice(c, b, q, rs, rp, 9, 1, 2, got=lists)
    check_attend(c, q, rs, rp, lists, 64)
