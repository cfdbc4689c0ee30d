"""Tree attention of batches that share prefixes, against the fp64 oracle.

Tolerances are those of tree attention: the arithmetic is the same but for the order of the sums, and the bound holds for any tree of
tiles.  A prefix and the own tokens are joined in fp32: two more products and a sum a part, inside the (log2 T + 16) u32 of the sum.
The groups share enough (cached tokens times key heads) for the prefix to be met together; where they do not, the call is plain tree
attention, which is tested too.
"""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.test_gpu_attention import U32, bf16, f64, i32, offsets, stored, tree_masks

pytestmark = pytest.mark.gpu


class Batch:
    """Groups of (requests' rows, own cached tokens) over `shared[g]` pages each; a filled cache."""

    def __init__(self, lib, seed, bits, groups, shared, hq, hk, d, page, masks="tree", qscale=1.5, spoil=None, pages_spare=2):
        r = np.random.default_rng(seed)
        self.lib, self.bits, self.hq, self.hk, self.d, self.page = lib, bits, hq, hk, d, page
        self.goffs, self.shared = offsets([len(g) for g in groups]), shared
        reqs = [(n, own, g) for g, list_ in enumerate(groups) for n, own in list_]
        self.counts = [n for n, _, _ in reqs]
        self.lens = [shared[g] * page + own for _, own, g in reqs]
        self.offs = offsets(self.counts)
        extra = [-(-(own + n) // page) for n, own, _ in reqs]
        n_pages = sum(shared) + sum(extra) + pages_spare
        perm = r.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(reqs), max(shared[g] + e for (_, _, g), e in zip(reqs, extra)) + 1), -5, np.int32)
        at, first = 0, []
        for g in range(len(groups)):
            first.append(perm[at:at + shared[g]])
            at += shared[g]
        for b, (_, _, g) in enumerate(reqs):
            self.table[b, :shared[g]] = first[g]
            self.table[b, shared[g]:shared[g] + extra[b]] = perm[at:at + extra[b]]
            at += extra[b]
        self.cache = lib.kv_cache_alloc(n_pages, page, hk, d, bits)
        for t in self.cache.tensors:                              # what no row may see: NaN everywhere
            t.fill_(float("nan")) if t.is_floating_point() else t.fill_(-1)
        fills = [(shared[g] * page, 0, b) for g in range(len(groups)) for b in [self.goffs[g]] if self.goffs[g + 1] > b]
        fills += [(own + n, shared[g] * page, b) for b, (n, own, g) in enumerate(reqs)]
        roff = offsets([f[0] for f in fills])
        k, v = bf16(r, roff[-1], hk * d), bf16(r, roff[-1], hk * d)
        if spoil:
            spoil(k, v, roff, len(fills) - len(reqs))
        tab = i32(np.ascontiguousarray(self.table[[f[2] for f in fills]]).tolist())
        for lo in range(0, len(fills), 200):
            hi = min(lo + 200, len(fills))
            s = slice(roff[lo], roff[hi])
            if roff[hi] > roff[lo]:
                lib.kv_append(self.cache, [o - roff[lo] for o in roff[lo:hi + 1]], i32([f[1] for f in fills[lo:hi]]), tab[lo:hi], k[s].cuda(), v[s].cuda())
        self.q = bf16(r, self.offs[-1], hq * d, scale=qscale)
        self.masks = tree_masks(r, self.counts) if masks == "tree" else masks
        self.mask = None if self.masks is None else torch.tensor([w - (1 << 64) if w >> 63 else w for w in self.masks], dtype=torch.int64, device="cuda")
        self.lens_d, self.table_d, self.q_d = i32(self.lens), i32(self.table.tolist()), self.q.cuda()
        self.groups = lib.prefix_groups(self.goffs, self.shared)
        assert lib.device_error() == 0

    def call(self, groups=None, **kw):
        return self.lib.tree_attention_shared(self.cache, groups or self.groups, self.offs, self.lens_d, self.table_d, self.q_d, self.hq, tree_mask=self.mask, **kw)

    def plain(self, **kw):
        return self.lib.tree_attention(self.cache, self.offs, self.lens_d, self.table_d, self.q_d, self.hq, tree_mask=self.mask, **kw)

    def shares(self):
        """Whether the call meets the prefix together: what it saves comes to 500,000 cached tokens times key heads."""
        rows = [sum(n > 0 for n in self.counts[lo:hi]) for lo, hi in zip(self.goffs, self.goffs[1:])]
        return sum(max(0, n - 1) * t for n, t in zip(rows, self.shared)) * self.page * self.hk >= 500000

    def check(self, got, scale=None, requests=None):
        scale = self.d ** -0.5 if scale is None else scale
        per, d, code = self.hq // self.hk, self.d, self.bits != 16
        for b in range(len(self.counts)) if requests is None else requests:
            m = self.counts[b]
            if not m:
                continue
            kk, vv = stored(self.cache, self.bits, self.table, self.page, b, self.lens[b] + m)
            mk = oa.chain_masks(m) if self.masks is None else self.masks[self.offs[b]:self.offs[b + 1]]
            seen = np.asarray(oa.visible(m, self.lens[b], mk)).astype(bool)
            rows = slice(self.offs[b], self.offs[b] + m)
            g, q = f64(got[rows]).reshape(m, self.hq, d), f64(self.q[rows]).reshape(m, self.hq, d)
            for h in range(self.hk):
                hs = slice(h * per, (h + 1) * per)
                qh, out, ok = q[:, hs].reshape(m * per, d), g[:, hs].reshape(m * per, d), np.repeat(seen, per, 0)
                k, v = np.where(seen.any(0)[:, None], kk[:, h], 0.0), np.where(seen.any(0)[:, None], vv[:, h], 0.0)
                # (a draft that some rows see and others do not may be anything but NaN or infinite here)
                z = np.where(ok, scale * (qh @ k.T), -np.inf)
                none = ~ok.any(1)
                assert (out[none] == 0).all()
                z[none] = 0.0
                p = np.exp(z - z.max(1, keepdims=True))
                p /= p.sum(1, keepdims=True)
                want = p @ v
                mag = abs(scale) * (np.abs(qh) @ np.abs(k).T)
                za = np.where(ok, np.abs(z), 0.0)
                e = mag * ((2.0 ** -11 if code else 0.0) + (d + 8) * U32) + 8 * U32 * (za + za.max(1, keepdims=True) + 1)
                rw = (2.0 ** -11 if code else 2.0 ** -8) + (np.log2(ok.sum(1, keepdims=True) + 1) + 16) * U32
                rr = rw + (2.0 ** -11 if code else 0.0)
                den = (p * np.expm1(e + rw)).sum(1, keepdims=True)
                assert (den[~none] < 0.5).all()
                bound = ((p * np.expm1(e + rr)) @ np.abs(v) + np.abs(want) * den) / (1 - den)
                bound = bound * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) + 1e-30
                err = np.abs(out - want)
                bad = (err > bound)[~none] | np.isnan(out)[~none]
                assert not bad.any(), (b, h, float((err / bound)[~none].max()))


ONES = [(1, i % 37) for i in range(64)]                           # a row each, over 0 .. 36 tokens of their own
MIXED = [(i % 13, (i * 7) % 50) for i in range(20)]               # requests without rows among them
SHAPES = [
    ([ONES], [63], 8, 8, 64, 16),                                 # 64 rows a key head: a block in both matrices
    ([MIXED], [130], 12, 4, 128, 64),                             # 342 rows: two blocks, the second of 86
    ([[(1, 5)] * 10, [(3, 200)], [], [(2, 0)] * 12, [(1, 1), (4, 17)]], [300, 40, 9, 200, 0], 8, 8, 64, 32),
    ([[(9, 300)] * 5], [245], 32, 2, 128, 256),                   # 720 rows: two full blocks and 208
    ([[(64, 100), (64, 3), (1, 0)]], [2100], 8, 8, 128, 16),      # 129 rows: one more than a matrix
    ([[(16, 0)] * 16], [33], 16, 16, 128, 64),                    # 256 rows: a full block; no own tokens but the drafts
    ([[(1, 0)] * 256], [123], 4, 1, 64, 16),                      # the most requests; a prefix that ends inside a tile
    ([[(1, 9)] * 2, [(2, 9)] * 2], [4097, 3001], 9, 9, 64, 16),
    ([[(2, 40)] * 8], [1], 4, 2, 64, 65536),                      # one page, the largest
    ([[(1, 3)] * 2] * 128, [40] * 128, 8, 8, 64, 16),             # 128 groups
    ([[(5, 20)] * 9], [245], 64, 1, 64, 256),                     # 64 query heads to a key head: twelve blocks
    ([[(2, 3)] * 3], [256], 4, 1, 64, 4096),                      # a million tokens
]


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_shared_prefixes(lib, bits, shape):
    groups, shared, hq, hk, d, page = SHAPES[shape]
    b = Batch(lib, 100 * shape + bits, bits, groups, shared, hq, hk, d, page, masks="tree" if shape % 2 == 0 else None)
    assert b.shares()
    rows = b.offs[-1]
    out = torch.full((rows + 1, hq * d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(lib.tree_attention_shared_workspace_bytes(b.cache, b.groups, b.offs, hq), dtype=torch.uint8, device="cuda")
    b.call(out=out, workspace=ws)
    assert lib.device_error() == 0
    assert (out[rows:] == 5.0).all() and (out[:, hq * d:] == 5.0).all() and not ws.any()
    some = sorted(set(range(0, len(b.counts), max(1, len(b.counts) // 12))) | {len(b.counts) - 1})
    b.check(out[:, :hq * d], requests=some)
    again = torch.zeros_like(out)
    b.call(out=again, workspace=ws)
    assert torch.equal(out[:rows, :hq * d], again[:rows, :hq * d])


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("scale", [0.17, -0.09, 0.0, 3.0])
def test_scales(lib, bits, scale):
    b = Batch(lib, 7 + bits, bits, [MIXED], [130], 4, 4, 64, 64, qscale=0.5)
    b.check(b.call(scale=scale), scale=scale, requests=[1, 12, 19])


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_far_scores(lib, bits):
    """References that move: in the prefix's first or last tile, or in the own tokens, lie scores that dwarf all others."""
    for where in ("first", "last", "own"):
        def spoil(k, v, roff, n):
            at = {"first": 3, "last": roff[1] - 2, "own": roff[n] + 4}[where]
            k[at] *= 30
        b = Batch(lib, 50 + bits, bits, [[(5, 40)] * 12], [190], 8, 4, 128, 64, qscale=4.0, spoil=spoil)
        assert b.shares()
        b.check(b.call(scale=0.02), scale=0.02, requests=[0, 5, 11])


@pytest.mark.parametrize("bits", [16, 8])
def test_masks_that_leave_no_draft(lib, bits):
    """A row that sees none of its request's drafts has the committed tokens; where there are none either but the prefix, that."""
    groups = [[(3, 0)] * 20, [(4, 20)] * 20]
    masks = [0, 0b10, 1 << 50] * 20 + [0, 0, 0b1000, ~0 & (1 << 64) - 1] * 20
    b = Batch(lib, 60, bits, groups, [120, 120], 8, 8, 64, 32, masks=masks)
    assert b.shares()
    b.check(b.call(), requests=[0, 7, 19, 20, 39])


@pytest.mark.parametrize("bits", [16, 8])
def test_values_that_are_not_finite_stay_with_those_that_see_them(lib, bits):
    """NaN and infinities in the own tokens of one request, in one group's prefix, and in drafts that no row sees."""
    groups = [[(4, 10)] * 16, [(4, 10)] * 16]

    def spoil(k, v, roff, n):
        k[roff[n + 3] + 2] = float("nan")                         # request 3's own tokens
        v[roff[n + 20] + 11], k[roff[n + 20] + 11] = float("inf"), float("-inf")   # request 20's draft 1, which no row sees
        v[roff[1] + 77, :64] = float("nan")                       # the second group's prefix, key head 0
    masks = [0b0001, 0b0001, 0b0101, 0b1001] * 32
    for i in range(32):
        masks[4 * i + 1] = 0b0001
    b = Batch(lib, 61, bits, groups, [150, 150], 8, 8, 64, 32, masks=masks, spoil=spoil)
    got = b.call()
    assert b.shares() and lib.device_error() == 0
    b.check(got, requests=[0, 2, 4, 15])
    assert got[12:16].isnan().any() and not got[:12].isnan().any() and not got[16:64].isnan().any()
    assert got[64:, :64].isnan().all() and not got[64:, 64:].isnan().any()


@pytest.mark.parametrize("bits", [16, 8])
def test_rows_of_q_that_are_not_finite_stay_alone(lib, bits):
    b = Batch(lib, 69, bits, [[(4, 10)] * 24], [100], 8, 8, 64, 32)
    assert b.shares()
    want = b.call()
    b.q_d[5, 64:128], b.q_d[30, 3] = float("nan"), float("inf")
    got = b.call()
    assert got[5, 64:128].isnan().all()
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[5, 64:128], keep[30, :64] = False, False
    assert torch.equal(got[keep], want[keep])


def test_in_place_and_strided_rows(lib):
    b = Batch(lib, 62, 16, [MIXED], [130], 4, 4, 128, 64)
    want = b.call()
    wide = torch.full((b.offs[-1] + 3, 4 * 128 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:b.offs[-1], 8:8 + 512] = b.q_d
    b.q_d = wide[:, 8:8 + 512]
    b.call(out=b.q_d)
    assert torch.equal(wide[:b.offs[-1], 8:520], want) and (wide[b.offs[-1]:] == 7.0).all() and (wide[:, :8] == 7.0).all() and (wide[:, 520:] == 7.0).all()


def test_small_savings_and_single_requests_are_plain_tree_attention(lib):
    for groups, shared in (([[(3, 5)] * 4], [10]), ([[(3, 5)], [(2, 9)]], [4000, 4000]), ([[(0, 5), (3, 5)]], [4000]), ([[(2, 5)] * 64], [0])):
        b = Batch(lib, 63, 16, groups, shared, 8, 8, 64, 16)
        assert not b.shares()
        assert torch.equal(b.call(), b.plain())


def test_the_groups_may_share_less_than_they_have(lib):
    """shared_pages below what the tables have in common, and groups split in two: the same rows within the bound."""
    b = Batch(lib, 64, 8, [[(2, 30)] * 32], [200], 8, 8, 64, 16)
    for goffs, shared in (([0, 32], [150]), ([0, 16, 32], [200, 160]), ([0, 0, 31, 32, 32], [0, 190, 200, 3])):
        g = lib.prefix_groups(goffs, shared)
        b.check(b.call(groups=g), requests=[0, 15, 16, 31])
    assert lib.device_error() == 0


def test_many_rows_over_a_short_prefix(lib):
    """More blocks than CTAs: 256 requests of 64 rows."""
    b = Batch(lib, 65, 16, [[(64, 0)] * 256], [16], 8, 8, 64, 16)
    assert b.shares()
    b.check(b.call(), requests=[0, 100, 255])


def test_largest_page_numbers(lib):
    """A cache past 2^31 elements and 4 GiB: its last pages hold the prefix."""
    n_pages, page, hk, d = 9000, 64, 32, 128                       # 2.36e9 elements each of K and V
    cache = lib.kv_cache(*[torch.zeros((n_pages, hk, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)])
    r = np.random.default_rng(66)
    B, pages = 16, 17
    table = np.zeros((B, pages + 1), np.int32)
    table[:, :pages] = n_pages - 1 - np.arange(pages)
    table[:, pages] = n_pages - 1 - pages - np.arange(B)
    T = pages * page
    k, v = bf16(r, T, hk * d), bf16(r, T, hk * d)
    lib.kv_append(cache, [0, T], i32([0]), i32(table[:1].tolist()), k.cuda(), v.cuda())
    k1, v1 = bf16(r, B, hk * d), bf16(r, B, hk * d)
    lens, tab, offs = i32([T] * B), i32(table.tolist()), list(range(B + 1))
    lib.kv_append(cache, offs, lens, tab, k1.cuda(), v1.cuda())
    q = bf16(r, B, hk * d).cuda()
    groups = lib.prefix_groups([0, B], [pages])
    got = lib.tree_attention_shared(cache, groups, offs, lens, tab, q, hk)
    kk = torch.cat([k.view(1, T, hk, d).expand(B, -1, -1, -1), k1.view(B, 1, hk, d)], 1).cuda().double()
    vv = torch.cat([v.view(1, T, hk, d).expand(B, -1, -1, -1), v1.view(B, 1, hk, d)], 1).cuda().double()
    z = torch.einsum("bhd,bthd->bht", q.double().view(B, hk, d), kk) * d ** -0.5
    p = z.softmax(-1)
    want = torch.einsum("bht,bthd->bhd", p, vv)
    # weights off by 2^-8 and by their exponents' (d + 8) u32 of at most 100, twice; the output's rounding
    bound = 2.1 * 2.0 ** -8 * torch.einsum("bht,bthd->bhd", p, vv.abs()) + 2.0 ** -8 * want.abs()
    assert ((got.double().view(B, hk, d) - want).abs() <= bound).all() and lib.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_bad_input_is_flagged(lib, bits):
    """A length inside the prefix, a page outside the cache: the error word says so and the other requests do not notice."""
    b = Batch(lib, 67, bits, [[(2, 30)] * 32, [(1, 3)] * 3], [200, 0], 8, 8, 64, 16)
    want = b.call()
    for what, value in (("len", 3199), ("len", 0), ("len", -1), ("len", 2 ** 31 - 1), ("own page", -1), ("own page", 1 << 30), ("prefix page", -7)):
        lens, table = b.lens_d.clone(), b.table_d.clone()
        if what == "len":
            lens[9] = value
        else:
            table[9 if what == "own page" else slice(0, 32), 200 if what == "own page" else 60] = value
        out = lib.tree_attention_shared(b.cache, b.groups, b.offs, lens, table, b.q_d, 8, tree_mask=b.mask)
        assert lib.device_error() == 4, what
        assert torch.equal(out[64:], want[64:])
        if what != "prefix page":
            assert torch.equal(out[:18], want[:18]) and torch.equal(out[20:], want[20:]), what
    assert torch.equal(b.call(), want) and lib.device_error() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_a_captured_call_follows_lengths_tables_and_queries(lib, bits):
    b = Batch(lib, 68, bits, [[(3, 60)] * 24], [90], 8, 8, 64, 32)
    assert b.shares()
    ws = torch.zeros(lib.tree_attention_shared_workspace_bytes(b.cache, b.groups, b.offs, 8), dtype=torch.uint8, device="cuda")
    out = b.call(workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.call(out=out, workspace=ws)
        b.call(out=out, workspace=ws)                              # one workspace, one call after the other
    full = b.lens_d.clone()
    for step in (0, 1, 2):
        b.lens_d.copy_(full - torch.arange(24, device="cuda", dtype=torch.int32) * step)
        b.q_d.mul_(0.5)
        b.table_d[:, :90] = b.table_d[:, :90].flip(1) if step == 2 else b.table_d[:, :90]
        g.replay()
        got = out.clone()
        assert torch.equal(got, b.call()) and not ws.any()
        ref = b.plain()
        # two results inside the bound of one: their weights' roundings apart, at most 2 (2^-8 + 2^-8) of the largest value
        assert ((got - ref).abs().float() <= 4 * 2.0 ** -8 * 4.5).all()
    assert lib.device_error() == 0


def test_two_streams_at_once(lib):
    bs = [Batch(lib, 70 + i, (16, 8)[i], [[(4, 50)] * 24], [100], 8, 8, 128, 32) for i in range(2)]
    want = [b.call() for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(6):
        for i in range(2):
            got[i].append(bs[i].call(stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
