"""Pages of a cache that requests share: fork, reserve, compact and page copies against the oracle's step-by-step state.

Everything here is integers and copies of bytes, so all comparisons are exact.
"""

import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests.test_gpu_attention import i32

pytestmark = pytest.mark.gpu


class World:
    """The GPU's state and caches beside the oracle's; every place of every page begins with contents of its own."""

    def __init__(self, lib, seed, n_pages, page, slots, width, layers=((2, 64, 16),)):
        self.lib, self.r, self.page, self.n_pages, self.slots = lib, np.random.default_rng(seed), page, n_pages, slots
        self.pages = lib.kv_pages_alloc(n_pages, page, slots, width)
        self.pages.block_table.fill_(-9)
        self.model = ot.Pages(n_pages, page, slots, width)
        self.model.table = [[-9] * width for _ in range(slots)]
        self.model.places = [[(p, i) for i in range(page)] for p in range(n_pages)]
        self.caches = [lib.kv_cache_alloc(n_pages, page, h, d, bits) for h, d, bits in layers]
        for c in self.caches:
            for t in c.tensors:
                raw = t.view(torch.int16)
                raw.copy_(torch.randint(-2 ** 15, 2 ** 15, raw.shape, dtype=torch.int16, device="cuda"))
        self.start = [[t.clone() for t in c.tensors] for c in self.caches]
        self.ws = torch.zeros(max(256, lib.kv_reserve_workspace_bytes(self.pages)), dtype=torch.uint8, device="cuda")

    def fork(self, parents, children, tokens):
        done = self.model.fork(parents, children, tokens)
        self.lib.kv_fork(self.pages, i32(parents), i32(children), i32(tokens))
        assert self.lib.device_error() == (0 if all(done) else 4)

    def reserve(self, keep, need, layers=True):
        missing, copies, fresh = self.model.reserve(keep, need)
        out = torch.full((self.slots, 3), -3, dtype=torch.int32, device="cuda")
        counts, out = self.lib.kv_reserve(self.pages, self.caches if layers else None, i32(keep), i32(need), copies=out, workspace=self.ws)
        assert counts.tolist() == [missing, len(copies), fresh], (keep, need)
        assert out.tolist() == [list(c) for c in copies] + [[-3] * 3] * (self.slots - len(copies))
        assert not self.ws.any() and self.lib.device_error() == 0
        return missing

    def compact(self):
        live, moves = self.model.compact()
        out = torch.full((self.n_pages, 2), -3, dtype=torch.int32, device="cuda")
        counts, out = self.lib.kv_compact(self.pages, self.caches, moves=out)
        assert counts.tolist() == [live, len(moves)]
        assert out.tolist() == [list(m) for m in moves] + [[-3] * 2] * (self.n_pages - len(moves)) and self.lib.device_error() == 0

    def check(self, contents=True):
        assert self.pages.refs.tolist() == self.model.refs and self.pages.held.tolist() == self.model.held
        table = self.pages.block_table.tolist()
        for s, n in enumerate(self.model.held):
            assert table[s][:n] == self.model.table[s][:n]
        if contents:
            src = torch.tensor([[p * self.page + i for p, i in row] for row in self.model.places], device="cuda")
            for c, old in zip(self.caches, self.start):
                for t, o in zip(c.tensors, old):
                    flat = o.view(torch.int16).transpose(1, 2).reshape(self.n_pages * self.page, o.shape[1], -1)   # [place, head, ...]
                    want = flat[src].transpose(1, 2)
                    assert torch.equal(t.view(torch.int16).reshape(want.shape), want)


def step(w, kv):
    """One random call; kv: the tokens that each slot keeps."""
    r, page = w.r, w.page
    kind = r.integers(0, 10)
    if kind < 2:
        live = [s for s in range(w.slots) if w.model.held[s]]
        empty = [s for s in range(w.slots) if not w.model.held[s]]
        n = int(r.integers(0, len(empty) + 1))
        if live and n:
            kids = [int(x) for x in r.choice(empty, n, replace=False)]
            par = [int(x) for x in r.choice(live, n)]
            tok = [int(r.integers(0, kv[p] + 1)) for p in par]
            w.fork(par, kids, tok)
            for c, t in zip(kids, tok):
                kv[c] = t
    elif kind == 2:
        w.compact()
    else:
        keep, need = [0] * w.slots, [-1] * w.slots
        for s in range(w.slots):
            act = r.integers(0, 6)
            if act < 3:
                keep[s] = kv[s]
                need[s] = kv[s] + int(r.integers(0, 3 * page if act else 9))
                need[s] = min(need[s], len(w.model.table[0]) * page)
            elif act == 3:
                keep[s] = need[s] = int(r.integers(0, kv[s] + 1))
            elif act == 4 and r.integers(0, 3) == 0:
                keep[s] = need[s] = 0
        before = list(kv)
        if not w.reserve(keep, need):
            kv[:] = [min(n, k + int(r.integers(0, max(1, n - k + 1)))) if n >= 0 else b for k, n, b in zip(keep, need, before)]


@pytest.mark.parametrize("seed,n_pages,page,slots,width,layers", [
    (1, 12, 16, 4, 5, [(2, 64, 16)]), (2, 40, 16, 9, 8, [(3, 128, 8)] * 2), (3, 100, 32, 20, 12, [(5, 192, 4)]),
    (4, 300, 64, 64, 9, [(2, 128, 16)]), (5, 90, 256, 33, 4, [(1, 256, 8)] * 3), (6, 1, 16, 1, 1, [(1, 64, 16)]),
    (7, 700, 16, 256, 7, [(1, 64, 8)]), (8, 33, 1024, 8, 6, [(1, 128, 4)])])
def test_random_calls(lib, seed, n_pages, page, slots, width, layers):
    w = World(lib, seed, n_pages, page, slots, width, layers)
    kv = [0] * slots
    for i in range(40):
        step(w, kv)
        if i % 5 == 4:
            w.check()
    w.check()


def test_many_layers_and_none(lib):
    """More caches than one launch takes, and bookkeeping alone."""
    w = World(lib, 9, 20, 16, 6, 6, [(1, 64, 8)] * 150)
    w.reserve([0] * 6, [70, -1, -1, -1, -1, -1])
    w.fork([0, 0, 0, 0], [1, 2, 3, 4], [70, 64, 40, 7])
    w.reserve([70, 64, 40, 7, 0, 0], [75, 70, 44, 7, -1, -1])
    w.check()
    w.reserve([0, 64, 40, 7, 0, 0], [0, 70, 40, 20, -1, -1])
    w.compact()
    w.check()
    a = World(lib, 10, 20, 16, 3, 6)
    a.caches, a.start = [], []
    a.reserve([0, 0, 0], [30, -1, -1], layers=False)
    a.fork([0], [1], [30])
    a.reserve([30, 30, 0], [40, 33, -1], layers=False)
    a.lib.kv_compact(a.pages, None)
    a.model.compact()
    a.check(contents=False)


def test_shortage_changes_nothing(lib):
    w = World(lib, 11, 6, 16, 4, 8)
    w.reserve([0] * 4, [40, 20, -1, -1])
    w.fork([0], [2], [40])
    before = [t.clone() for t in (w.pages.refs, w.pages.block_table, w.pages.held)]
    assert w.reserve([40, 0, 33, 0], [41, 0, 100, -1]) > 0          # what slot 1 gives back is not free before the call
    assert all(torch.equal(a, b) for a, b in zip(before, (w.pages.refs, w.pages.block_table, w.pages.held)))
    w.check()
    assert w.reserve([40, 0, 33, 0], [40, 0, 33, -1]) == 0


@pytest.mark.parametrize("fill", [0x7f, 0xff, 1])
def test_the_workspace_may_hold_anything(lib, fill):
    for keep, need in (([40, 20, 0, 0], [-1, -1, -1, -1]), ([40, 20, 33, 0], [41, -1, 100, -1]), ([49, 20, 0, 0], [50, 10, -1, 30]), ([8, 0, 33, 0], [8, 0, 40, 16])):
        w = World(lib, 18, 8, 16, 4, 8)
        w.reserve([0] * 4, [40, 20, -1, -1])
        w.fork([0], [2], [40])
        ws = torch.full_like(w.ws, fill)
        bad = [k > n >= 0 or k > 16 * h for k, n, h in zip(keep, need, w.model.held)]
        want = w.model.reserve([0 if x else k for k, x in zip(keep, bad)], [-1 if x else n for n, x in zip(need, bad)])
        counts, _ = lib.kv_reserve(w.pages, w.caches, i32(keep), i32(need), workspace=ws)
        assert counts.tolist() == [want[0], len(want[1]), want[2]] and lib.device_error() == (4 if any(bad) else 0)
        w.check()


def test_bad_forks_and_reserves_are_flagged_and_alone(lib):
    for bad in [dict(parent=-1), dict(parent=6), dict(child=-2), dict(child=6), dict(child=1), dict(child=0), dict(tokens=-1), dict(tokens=49),
                dict(child=3), dict(tokens=2 ** 31 - 1)]:
        w = World(lib, 12, 12, 16, 6, 4)
        w.reserve([0] * 6, [48, 5, -1, -1, -1, -1])
        call = dict(parent=0, child=2, tokens=17)
        call.update(bad)
        w.fork([0, call["parent"]], [3, call["child"]], [48, call["tokens"]])
        w.check(contents=False)
    w = World(lib, 13, 12, 16, 6, 4)
    w.reserve([0] * 6, [48, 5, -1, -1, -1, -1])
    w.fork([0, 2, 1], [2, 3, 4], [48, 16, 5])                       # a child that is another's parent: neither works from the other
    w.check(contents=False)
    for keep, need in ((49, 60), (-1, 5), (6, 5), (48, 65), (0, 2 ** 31 - 1)):
        w = World(lib, 14, 12, 16, 3, 4)
        w.reserve([0] * 3, [48, 5, -1])
        counts, _ = lib.kv_reserve(w.pages, w.caches, i32([keep, 5, 0]), i32([need, 20, -1]))
        assert lib.device_error() == 4 and counts.tolist() == [0, 0, 1]
        w.model.reserve([0, 5, 0], [-1, 20, -1])
        w.check()


def test_pages_out_of_range_are_flagged(lib):
    for page in (-1, 12, 2 ** 31 - 1):
        w = World(lib, 15, 12, 16, 3, 4)
        w.reserve([0] * 3, [48, 5, -1])
        w.pages.block_table[0, 1] = page
        lib.kv_fork(w.pages, i32([0, 1]), i32([2, 2]), i32([48, 5]))
        assert lib.device_error() == 4
        lib.kv_reserve(w.pages, w.caches, i32([20, 5, 0]), i32([40, 6, -1]))
        assert lib.device_error() == 4
        refs = w.pages.refs.clone()
        counts, _ = lib.kv_compact(w.pages, w.caches)
        assert lib.device_error() == 4 and counts.tolist() == [int((refs > 0).sum()), 0]
        assert w.pages.block_table[0, 1].item() == page


@pytest.mark.parametrize("bits,heads,dim,page", [(16, 1, 64, 16), (16, 8, 128, 64), (8, 3, 192, 16), (4, 1, 64, 16), (4, 5, 256, 128), (8, 2, 64, 512)])
def test_copy_pages(lib, bits, heads, dim, page):
    r = np.random.default_rng(bits + dim)

    def cache(n):
        c = lib.kv_cache_alloc(n, page, heads, dim, bits)
        for t in c.tensors:
            raw = t.view(torch.int16)
            raw.copy_(torch.randint(-2 ** 15, 2 ** 15, raw.shape, dtype=torch.int16, device="cuda"))
        return c
    for n, layers in ((1, 1), (37, 3), (90, 70)):
        a, b = [cache(95) for _ in range(layers)], [cache(200) for _ in range(layers)]
        keep = [[t.clone() for t in c.tensors] for c in b]
        src, dst = r.integers(0, 95, n), r.permutation(200)[:n]
        lib.kv_copy_pages(a, i32(src.tolist()), i32(dst.tolist()), to=b)
        for c, o, k in zip(a, b, keep):
            for t, u, v in zip(c.tensors, o.tensors, k):
                v[torch.from_numpy(dst)] = t[torch.from_numpy(src)]
                assert torch.equal(u.view(torch.int16), v.view(torch.int16))
        pair = r.permutation(95)
        keep = [[t.clone() for t in c.tensors] for c in a]
        lib.kv_copy_pages(a, i32(pair[:n // 2].tolist()), i32(pair[n // 2:2 * (n // 2)].tolist()))
        for c, k in zip(a, keep):
            for t, v in zip(c.tensors, k):
                v[torch.from_numpy(pair[n // 2:2 * (n // 2)])] = v[torch.from_numpy(pair[:n // 2])]
                assert torch.equal(t.view(torch.int16), v.view(torch.int16))
    assert lib.device_error() == 0
    keep = [t.clone() for t in a[0].tensors]
    lib.kv_copy_pages(a[:1], i32([0, 95, -1, 3, 2 ** 31 - 1]), i32([1, 2, 4, 95, 5]))
    assert lib.device_error() == 4
    for t, v in zip(a[0].tensors, keep):
        v[1] = v[0]
        assert torch.equal(t.view(torch.int16), v.view(torch.int16))
    lib.kv_copy_pages(a, i32([]), i32([]))


def test_largest_pages(lib):
    """Pages of 65536 tokens: copied whole, moved, and in part."""
    w = World(lib, 19, 4, 65536, 3, 2, [(2, 64, 4)] * 2)
    w.reserve([0] * 3, [40001, 65537, -1])
    w.fork([0], [2], [40001])
    w.reserve([0, 0, 40001], [-1, 0, 50000])                        # (slot 0 is left alone: its page stays shared until then)
    w.check()
    w.reserve([0, 0, 0], [0, -1, -1])
    w.compact()
    w.check()
    lib.kv_copy_pages(w.caches, i32([0]), i32([3]))
    assert all(torch.equal(t[3].view(torch.int16), t[0].view(torch.int16)) for c in w.caches for t in c.tensors) and lib.device_error() == 0


def test_offsets_past_32_bits(lib):
    """A cache of more than 2^32 bytes a tensor: its last page."""
    n, heads, page, dim = 9000, 32, 64, 128
    c = lib.kv_cache(*[torch.zeros((n, heads, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    c.k[n - 1], c.v[n - 1] = 3.0, 4.0
    lib.kv_copy_pages([c], i32([n - 1, n - 1]), i32([n - 2, 7]))
    for p in (n - 2, 7):
        assert (c.k[p] == 3).all() and (c.v[p] == 4).all()
    pages = lib.kv_pages_alloc(n, page, 2, 4)
    pages.refs[:n - 1] = 1
    pages.refs[n - 1], pages.refs[n - 3] = 2, 0
    pages.block_table[:, 0], pages.held[:] = n - 1, 1
    counts, copies = lib.kv_reserve(pages, [c], i32([40, 0]), i32([50, -1]))
    assert counts.tolist() == [0, 1, 1] and copies[0].tolist() == [n - 1, n - 3, 40] and (c.k[n - 3, :, :40] == 3).all() and not c.v[n - 3, :, 40:].any()
    pages.refs[:] = 0
    pages.refs[n - 1] = 1
    pages.held[0] = 0
    counts, moves = lib.kv_compact(pages, [c])
    assert counts.tolist() == [1, 1] and moves[0].tolist() == [n - 1, 0] and (c.v[0] == 4).all() and pages.block_table[1, 0].item() == 0
    assert lib.device_error() == 0


def test_largest_states(lib):
    """A hundred thousand pages, 256 slots of long tables."""
    w = World(lib, 16, 100003, 16, 256, 2000, layers=())
    w.caches = None
    need = [int(x) for x in w.r.integers(0, 12000, 256)]
    keep = [0] * 256
    w.model.places = [[]] * w.n_pages
    w.model.page = 16
    missing, copies, fresh = w.model.reserve(keep, need)
    counts, _ = lib.kv_reserve(w.pages, None, i32(keep), i32(need))
    assert counts.tolist() == [missing, 0, fresh] and missing == 0
    w.check(contents=False)
    half = [n // 2 if i % 3 else 0 for i, n in enumerate(need)]
    assert lib.kv_reserve(w.pages, None, i32(half), i32(half))[0].tolist() == [0, 0, 0]
    w.model.reserve(half, half)
    w.check(contents=False)
    live, moves = w.model.compact()
    counts, out = lib.kv_compact(w.pages, None)
    assert counts.tolist() == [live, len(moves)] and out[:len(moves)].tolist() == [list(m) for m in moves]
    w.check(contents=False)


def test_a_captured_round_replays_as_the_state_changes(lib):
    w = World(lib, 17, 40, 16, 5, 8, [(2, 64, 8)])
    w.reserve([0] * 5, [50, -1, -1, -1, -1])
    keep, need, par, kid, tok = i32([0] * 5), i32([-1] * 5), i32([0, 0]), i32([1, 2]), i32([50, 50])
    counts, copies, moves = i32([0] * 3), torch.zeros((5, 3), dtype=torch.int32, device="cuda"), torch.zeros((40, 2), dtype=torch.int32, device="cuda")
    live = i32([0, 0])
    warm = lib.kv_pages_alloc(40, 16, 5, 8)
    lib.kv_reserve(warm, w.caches, keep, need, counts=counts, copies=copies, workspace=w.ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.kv_fork(w.pages, par, kid, tok)
        lib.kv_reserve(w.pages, w.caches, keep, need, counts=counts, copies=copies, workspace=w.ws)
        lib.kv_compact(w.pages, w.caches, counts=live, moves=moves)
    for k, n, p, c, t in (([50, 50, 50, 0, 0], [60, 55, 70, -1, -1], [0, 0], [1, 2], [50, 50]),
                          ([10, 55, 0, 60, 20], [10, 56, 0, 64, 30], [1, 0], [4, 3], [20, 60]),
                          ([10, 56, 0, 0, 30], [100, 56, -1, 0, 31], [0, 0], [2, 2], [1, 1])):
        ok = w.model.fork(p, c, t)
        want = w.model.reserve(k, n)
        assert want[0] == 0
        moved = w.model.compact()
        for a, v in ((keep, k), (need, n), (par, p), (kid, c), (tok, t)):
            a.copy_(i32(v))
        g.replay()
        torch.cuda.synchronize()
        assert lib.device_error() == (0 if all(ok) else 4)
        assert counts.tolist() == [0, len(want[1]), want[2]] and live.tolist() == [moved[0], len(moved[1])]
        w.check()
