"""The 4-bit store, the weight and the cut from several host threads on streams of their own, and as graphs that are
replayed in turn: each caller's answer is what it gets alone."""

import threading

import numpy as np
import pytest
import torch

from paged_kv_cache_235_gb300 import binding as B
from tests import gpu64 as X

pytestmark = pytest.mark.gpu

L = [17001, 9000, 700]


class Server:
    """A cache and the calls of one step on it: store, decode, weight; and a cut of every stream to half."""

    def __init__(self, kv, seed):
        self.c = c = X.LongCase(kv, L, [True, False, True], 8, 2, seed)
        self.rs, self.rp = X.last_rows(L, [1, 2, 1])
        self.q = c.q(4)
        self.k, self.v = (torch.randn(4, 2, 128, generator=c.g, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.out, self.lse = torch.empty(4, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 8, device="cuda")
        self.back = [torch.empty(4, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.mass, self.moves = torch.zeros(3, 2, 17004, device="cuda"), B.make_moves(3, 2, 17004)
        self.sc = B.make_scratch(4, 8)
        self.keep = np.array([n // 2 for n in L], np.int32)

    def step(self, stream=None):
        c = self.c
        B.tfpa_write_kv(c.cache, c.segs, self.k, self.v, self.rs, self.rp, stream=stream)
        B.tfpa_read_kv(c.cache, c.segs, *self.back, self.rs, self.rp, stream=stream)
        B.tfpa_decode(c.cache, c.segs, self.q, self.rs, self.rp, X.SCALE, self.sc, self.out, self.lse, stream=stream)
        B.tfpa_key_mass(c.cache, c.segs, self.q, self.lse, self.rs, self.rp, X.SCALE, self.mass, decay=0.5, stream=stream)

    def cut(self, stream=None):
        B.tfpa_evict_kv(self.c.cache, self.c.segs, self.keep, self.mass, self.moves, sink=4, recent=64, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        assert int(self.c.err.item()) == 0
        return [self.out, self.lse, *self.back, self.mass, self.moves[..., 0], self.c.k_pool.view(torch.uint8), self.c.v_pool.view(torch.uint8),
                *[t.view(torch.uint8) for s in self.c.slabs.values() for t in s]]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a.state(), b.state()))


def test_threads_on_streams_of_their_own():
    kvs = ["fp4", "bf16", "fp8", "fp4"]
    servers, alone = [Server(kv, 160 + i) for i, kv in enumerate(kvs)], [Server(kv, 160 + i) for i, kv in enumerate(kvs)]
    torch.cuda.synchronize()
    errors = []

    def work(s):
        try:
            st = torch.cuda.Stream()
            for _ in range(8):
                s.step(st)
            s.cut(st)
            st.synchronize()
        except Exception as e:                                   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(s,)) for s in servers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for s, a in zip(servers, alone):
        for _ in range(8):
            a.step()
        a.cut()
        assert same(s, a)


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_graphs_of_two_caches_replayed_in_turn(kv):
    """Long streams, so the cut's choice runs in clusters."""
    servers, alone = [Server(kv, 170 + i) for i in range(2)], [Server(kv, 170 + i) for i in range(2)]
    torch.cuda.synchronize()
    stream, graphs = torch.cuda.Stream(), []
    for s in servers:
        pair = []
        for fn in (s.step, s.cut):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                fn()
            pair.append(g)
        graphs.append(pair)
    for _ in range(3):
        for step, _cut in graphs:
            step.replay()
    for _step, cut in graphs:
        cut.replay()
    for a in alone:
        for _ in range(3):
            a.step()
        a.cut()
    for s, a in zip(servers, alone):
        assert same(s, a)
