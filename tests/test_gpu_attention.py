"""The attention-side calls against the fp64 oracle, at the sizes, masks and layouts where they can go wrong.

Tolerances, from the arithmetic (u = half a step: bf16 2^-8, fp16 2^-11, fp32 2^-24 relative to the value):

* norm and rotation: one bf16 rounding of the output, 2^-8 |y|, plus fp32 work on the pair: the mean's sum and
  the products take under 24 fp32 roundings and the angle is off by at most 2 pi 2^-25 + 2^-24 rad, so
  32 u32 (|x_i| + |x_j|) covers them.
* cache: codes, scales and biases are equal to the last bit (the format's roundings are IEEE fp32 and fp16); read back
  values carry one fp32 and one bf16 rounding.
* attention: with e_t the error of the exponent of token t, w the relative error of a weight and r that of a weight and a
  value together, out_d moves by at most  (sum_t p_t |v_td| x_t + |out_d| sum_t p_t y_t) / (1 - sum_t p_t y_t),
  x_t = exp(r + e_t) - 1, y_t = exp(w + e_t) - 1: the sum of the weights may be taken before or after their rounding.
  e_t: for codes, K enters the product as fp16 (2^-11 per element) - scale sum_d |q_d k_td| 2^-11 - and fp32
  accumulation adds (dim + 8) u32 of the same sum; the exponent itself (a product and a subtraction in fp32 and the
  hardware exponential, 2^-22) adds 8 u32 (|score| + 1).  w: the weight is rounded to 16 bits, 2^-8 over a bf16
  cache and 2^-11 over codes; V enters as fp16 over codes (another 2^-11); the sum over T tokens in fp32 adds
  (log2 T + 16) u32 in any tree of 128-token tiles.  Last, one bf16 rounding of the output.
"""

import math

import numpy as np
import pytest
import torch

from oracle import attention as oa
from speculative_decoding_verify_qmm_gb300.binding import SVError

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def bf16(r, *shape, scale=1.0):
    return torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ norm and rotation

def check_rope(got, x, weight, norm, pos, inv, interleaved):
    want = oa.norm_rope(x, weight, 1e-6, norm, pos, inv, interleaved)
    half = 0 if inv is None else len(inv)
    plain = np.abs(oa.norm_rope(x, weight, 1e-6, norm, None, None, False))
    both = plain.copy()
    if half:
        i = slice(0, 2 * half, 2) if interleaved else slice(0, half)
        j = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
        s = plain[..., i] + plain[..., j]
        both[..., i], both[..., j] = s, s
    bound = 2.0 ** -8 * np.abs(want) + 32 * U32 * both + 1e-38
    err = np.abs(got - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("rows,hq,hk,d,rot,interleaved,norm", [
    (1, 1, 1, 64, 64, False, True), (8, 32, 8, 128, 128, False, True), (8, 32, 8, 128, 128, True, True),
    (3, 5, 1, 128, 32, False, False), (3, 6, 2, 96, 96, True, True), (2, 3, 1, 80, 48, False, True),
    (2, 1, 0, 8, 0, False, True), (2, 4, 4, 256, 256, False, True), (5, 48, 8, 128, 96, False, True),
    (400, 7, 3, 128, 128, False, True), (1, 33, 17, 16, 16, True, False), (311, 48, 8, 128, 64, True, True)])
def test_norm_rope(lib, rows, hq, hk, d, rot, interleaved, norm):
    r = np.random.default_rng(rows * 1000 + d)
    qkv = bf16(r, rows + 2, (hq + 2 * max(hk, 1)) * d, scale=3.0).cuda()
    qw, kw = (1 + bf16(r, d, scale=0.2)).cuda(), (1 + bf16(r, d, scale=0.2)).cuda()
    pos = r.integers(0, 1000000, rows)
    inv = (1e6 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    q, k = qkv[:rows, :hq * d], (qkv[:rows, hq * d:(hq + hk) * d] if hk else None)
    args = dict(positions=i32(pos.tolist()), inv_freq=torch.from_numpy(inv).cuda()) if rot else {}
    qo, ko = lib.qk_norm_rope(q, k, d, q_weight=qw, k_weight=kw, norm=norm, interleaved=interleaved, **args)
    for out, x, w, n in ((qo, q, qw, hq), (ko, k, kw, hk)):
        if n:
            check_rope(f64(out).reshape(rows, n, d), f64(x).reshape(rows, n, d), f64(w), norm, pos, inv if rot else None,
                       interleaved)
    # in place, inside the projection's output: the same values, and nothing else touched
    before = qkv.clone()
    lib.qk_norm_rope(q, k, d, q_weight=qw, k_weight=kw, norm=norm, interleaved=interleaved, q_out=q, k_out=k, **args)
    assert torch.equal(q, qo) and (not hk or torch.equal(k, ko))
    assert torch.equal(qkv[rows:], before[rows:]) and torch.equal(qkv[:, (hq + hk) * d:], before[:, (hq + hk) * d:])


def test_norm_rope_unaligned_and_weightless(lib):
    r = np.random.default_rng(7)
    rows, hq, hk, d = 3, 4, 2, 64
    buf = bf16(r, rows, (hq + hk) * d + 5).cuda()
    q, k = buf[:, 1:1 + hq * d], buf[:, 3 + hq * d:3 + (hq + hk) * d]        # odd offsets, an odd stride
    pos, inv = [0, 5, -7], (1e4 ** (-np.arange(32) / 32)).astype(np.float32)
    qo, ko = lib.qk_norm_rope(q, k, d, i32(pos), torch.from_numpy(inv).cuda())
    check_rope(f64(qo).reshape(rows, hq, d), f64(q).reshape(rows, hq, d), None, True, pos, inv, False)
    check_rope(f64(ko).reshape(rows, hk, d), f64(k).reshape(rows, hk, d), None, True, pos, inv, False)


def test_norm_rope_keeps_rows_apart(lib):
    r = np.random.default_rng(8)
    x = bf16(r, 4, 2 * 64).cuda()
    want, _ = lib.qk_norm_rope(x, None, 64)
    y = x.clone()
    y[1, 3], y[2, 70] = float("nan"), float("inf")
    got, _ = lib.qk_norm_rope(y, None, 64)
    assert torch.equal(got[[0, 3]], want[[0, 3]]) and torch.equal(got[1, 64:], want[1, 64:])
    assert got[1, :64].isnan().all() and torch.equal(got[2, :64], want[2, :64])
    empty, _ = lib.qk_norm_rope(x[:0], None, 64)
    assert empty.shape == (0, 128)


# ------------------------------------------------------------------- the cache

def tables(r, spans, page, spare=2):
    """Shuffled pages for `spans` tokens a request; entries past the last used page hold an invalid page."""
    n = [-(-max(1, s) // page) for s in spans]
    perm = r.permutation(sum(n) + spare).astype(np.int32)
    t = np.full((len(spans), max(n) + 1), -5, dtype=np.int32)
    at = 0
    for b, c in enumerate(n):
        t[b, :c] = perm[at:at + c]
        at += c
    return t, sum(n) + spare


def offsets(counts):
    return [0] + np.cumsum(counts).tolist()


def stored(cache, bits, table, page, b, n):
    """fp64 (k, v) [n, heads, dim] of request b's first n positions, from the cache's own tensors."""
    out = []
    t = [x.cpu().numpy() if bits != 16 or i > 1 else f64(x) for i, x in enumerate(cache.tensors)]
    pages, at = table[b, np.arange(n) // page], np.arange(n) % page
    for i in range(2):
        x = t[i][pages, :, at]
        if bits != 16:
            x = oa.kv_dequantize(oa.unpack(x.view(np.uint32), bits), t[2 + 2 * i][pages, :, at], t[3 + 2 * i][pages, :, at])
        out.append(x)
    return out


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("counts,lens,hk,d,page", [
    ([1], [0], 1, 64, 16), ([3, 0, 17], [15, 4, 30], 2, 128, 16), ([40, 1], [0, 127], 8, 128, 64),
    ([5, 33, 2, 1], [1, 2, 3, 63], 3, 192, 32), ([300], [11], 1, 256, 128)])
def test_append_and_read(lib, bits, counts, lens, hk, d, page):
    r = np.random.default_rng(sum(counts) * 10 + bits)
    offs = offsets(counts)
    table, n_pages = tables(r, [n + c for n, c in zip(lens, counts)], page)
    cache = lib.kv_cache_alloc(n_pages, page, hk, d, bits)
    for t in cache.tensors:
        t.fill_(3)
    before = [t.clone() for t in cache.tensors]
    x = bf16(r, offs[-1] + 2, 3 * hk * d + 8, scale=2.0)
    x[0, :64] = 0.75                                                        # a flat group
    x = x.cuda()
    k, v = x[:, :hk * d], x[:, 2 * hk * d:3 * hk * d]
    lib.kv_append(cache, offs, i32(lens), i32(table.tolist()), k, v)
    # expected tensors: only the new rows' places differ from what was there
    want = [t.cpu() for t in before]
    for b in range(len(counts)):
        for i in range(counts[b]):
            pos = lens[b] + i
            pg, at, row = int(table[b, pos // page]), pos % page, offs[b] + i
            for s, src in enumerate((k, v)):
                vec = src[row].cpu().reshape(hk, d)
                if bits == 16:
                    want[s][pg, :, at] = vec
                else:
                    c, sc, bi = oa.kv_quantize(vec.float().numpy(), bits)
                    want[s][pg, :, at] = torch.from_numpy(oa.pack(c, bits).view(np.int32))
                    want[2 + 2 * s][pg, :, at] = torch.from_numpy(sc)
                    want[3 + 2 * s][pg, :, at] = torch.from_numpy(bi)
    for got, w in zip(cache.tensors, want):
        assert torch.equal(got.cpu(), w)
    ko, vo = (torch.full((offs[-1] + 2, hk * d + 8), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lib.kv_read(cache, offs, i32(lens), i32(table.tolist()), k=ko, v=vo)
    for s, out in enumerate((ko, vo)):
        assert torch.all(out[offs[-1]:] == 9.0) and torch.all(out[:, hk * d:] == 9.0)
        for b in range(len(counts)):
            ref = stored(cache, bits, table, page, b, lens[b] + counts[b])[s][lens[b]:]
            got = f64(out[offs[b]:offs[b + 1], :hk * d]).reshape(ref.shape)
            assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 4 * U32 * np.abs(ref) + 1e-38)
    assert lib.device_error() == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_append_far_values_and_nan(lib, bits):
    r = np.random.default_rng(11)
    x = bf16(r, 4, 128)
    x[0, 5], x[0, 7], x[1, 70], x[2, 3] = float("inf"), -3e38, float("nan"), 1e-30
    x[3, :64] = torch.linspace(-1e-5, 1e-5, 64).to(torch.bfloat16)          # scales below fp16's normal range
    x = x.cuda()
    cache = lib.kv_cache_alloc(2, 16, 1, 128, bits)
    lib.kv_append(cache, [0, 4], i32([0]), i32([[1]]), x, x)
    c, s, b = oa.kv_quantize(x.cpu().float().numpy(), bits)
    assert torch.equal(cache.k[1, 0, :4].cpu(), torch.from_numpy(oa.pack(c, bits).view(np.int32)))
    assert np.array_equal(cache.tensors[2][1, 0, :4].cpu().numpy(), s, equal_nan=True)
    k, v = lib.kv_read(cache, [0, 4], i32([0]), i32([[1]]))
    assert k[1, 64:].isnan().all() and not k[1, :64].isnan().any() and k[0].isfinite().all()
    assert torch.equal(k.nan_to_num(7.0), v.nan_to_num(7.0))


def test_unaligned_rows(lib):
    r = np.random.default_rng(12)
    x = bf16(r, 5, 2 * 64 + 3).cuda()
    for bits in (16, 8, 4):
        a, b = lib.kv_cache_alloc(1, 16, 2, 64, bits), lib.kv_cache_alloc(1, 16, 2, 64, bits)
        lib.kv_append(a, [0, 5], i32([2]), i32([[0]]), x[:, 1:129], x[:, 3:131])
        lib.kv_append(b, [0, 5], i32([2]), i32([[0]]), x[:, 1:129].contiguous(), x[:, 3:131].contiguous())
        assert all(torch.equal(s, t) for s, t in zip(a.tensors, b.tensors))
        ko, vo = torch.zeros_like(x), torch.zeros_like(x)
        lib.kv_read(a, [0, 5], i32([2]), i32([[0]]), k=ko[:, 1:129], v=vo[:, 3:131])
        kc, vc = lib.kv_read(a, [0, 5], i32([2]), i32([[0]]))
        assert torch.equal(ko[:, 1:129], kc) and torch.equal(vo[:, 3:131], vc)


@pytest.mark.parametrize("bits", [16, 8])
def test_bad_pages_and_lengths_are_flagged(lib, bits):
    """A page outside the cache, a negative length and a position past the table: nothing is written, the error word says so."""
    r = np.random.default_rng(13)
    x = bf16(r, 6, 64).cuda()
    cache = lib.kv_cache_alloc(3, 16, 1, 64, bits)
    lib.device_error()
    for lens, table in [([14, 0, 0], [[0, 3], [1, -1], [2, -1]]), ([0, -1, 0], [[0, 1], [1, -1], [2, -1]]),
                        ([31, 0, 0], [[0, 1], [1, -1], [2, -1]]), ([2 ** 31 - 1, 0, 0], [[0, 1], [1, -1], [2, -1]])]:
        for t in cache.tensors:
            t.zero_()
        lib.kv_append(cache, [0, 4, 5, 6], i32(lens), i32(table), x, x)
        assert lib.device_error() == 4
        ko, vo = (torch.full((6, 64), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        lib.kv_read(cache, [0, 4, 5, 6], i32(lens), i32(table), k=ko, v=vo)
        assert lib.device_error() == 4
        good = [lens[0] + i >= 0 and (lens[0] + i) // 16 < 2 and 0 <= table[0][(lens[0] + i) // 16] < 3 for i in range(4)] \
            + [lens[1] >= 0, lens[2] >= 0]
        for i, g in enumerate(good):
            assert torch.all(ko[i] == 9.0).item() != g
        if bits == 16:
            assert torch.equal(ko[good], x[good])
    assert lib.device_error() == 0


# --------------------------------------------------------------------- commit

@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("layers,hk,d,page", [(1, 1, 64, 16), (3, 2, 128, 16), (70, 2, 64, 32)])
def test_commit(lib, bits, layers, hk, d, page):
    r = np.random.default_rng(bits + layers)
    m = [64, 9, 1, 33]
    paths = [[0] + sorted(r.choice(np.arange(1, 64), 20, replace=False).tolist()), [0, 1, 2], [0], [3, 4, 30]]
    lens = [7, 0, 40, 29]
    table, n_pages = tables(r, [a + b for a, b in zip(lens, m)], page)
    caches = [lib.kv_cache_alloc(n_pages, page, hk, d, bits) for _ in range(layers)]
    for c in caches:
        for t in c.tensors:
            t.copy_(torch.from_numpy(r.integers(0, 255, tuple(t.shape))).to(t.dtype))
    before = [[t.clone() for t in c.tensors] for c in caches]
    pm = np.full((4, 25), -9, dtype=np.int32)
    for b, p in enumerate(paths):
        pm[b, :len(p)] = p
    lib.kv_commit(caches, i32(lens), i32(table.tolist()), i32(pm.tolist()), i32([len(p) for p in paths]))
    assert lib.device_error() == 0
    for c, old in zip(caches, before):
        for t, o in zip(c.tensors, old):
            want = o.clone()
            for b, p in enumerate(paths):
                n = lens[b] + m[b]
                src = oa.commit(np.arange(n), lens[b], p)
                pos = np.arange(n)
                pg, at = torch.from_numpy(table[b, pos // page].astype(np.int64)), torch.from_numpy(pos % page)
                sg, st = pg[torch.from_numpy(src)], at[torch.from_numpy(src)]
                want[pg, :, at] = o[sg, :, st]
            assert torch.equal(t, want)


def test_commit_flags_bad_paths_and_leaves_the_request(lib):
    r = np.random.default_rng(15)
    cache = lib.kv_cache_alloc(4, 16, 1, 64, 16)
    cache.k.copy_(bf16(r, 4, 1, 16, 64))
    before = cache.k.clone()
    table = i32([[0, 1], [2, 3]])
    lib.device_error()
    for path, n, lens in [([2, 1], 2, 3), ([0, 0], 2, 3), ([0, 64], 2, 3), ([-1, 2], 2, 3), ([0, 5], 3, 3), ([0, 5], -1, 3),
                          ([0, 30], 2, 3), ([0, 5], 2, -1)]:
        cache.k.copy_(before)
        lib.kv_commit([cache], i32([lens, 1]), table, i32([path, [0, 4]]), i32([n, 2]))
        assert lib.device_error() == 4
        assert torch.equal(cache.k[:2], before[:2])
        assert torch.equal(cache.k[2, :, 2], before[2, :, 5])                 # the other request is served
    cache.k.copy_(before)
    lib.kv_commit([cache], i32([3, 1]), table, i32([[5, 9], [5, 9]]), i32([0, 0]))
    assert torch.equal(cache.k, before) and lib.device_error() == 0


# ------------------------------------------------------------------ attention

def attend_case(lib, r, bits, counts, lens, hq, hk, d, page, masks=None, qscale=1.5, spoil=None):
    """A filled cache and its call's arguments; `spoil` edits the bf16 rows (per request: k, v) before they are stored."""
    offs = offsets(counts)
    spans = [n + c for n, c in zip(lens, counts)]
    table, n_pages = tables(r, spans, page)
    cache = lib.kv_cache_alloc(n_pages, page, hk, d, bits)
    for t in cache.tensors:                                                  # what no row may see: NaN everywhere
        t.fill_(float("nan")) if t.is_floating_point() else t.fill_(-1)
    roff = offsets(spans)
    k, v = bf16(r, roff[-1], hk * d), bf16(r, roff[-1], hk * d)
    if spoil:
        spoil(k, v, roff)
    if roff[-1]:
        lib.kv_append(cache, roff, i32([0] * len(counts)), i32(table.tolist()), k.cuda(), v.cuda())
    q = bf16(r, offs[-1], hq * d, scale=qscale)
    mask = None
    if masks is not None:
        mask = torch.tensor([w - (1 << 64) if w >> 63 else w for w in masks], dtype=torch.int64, device="cuda")
    return cache, offs, table, q, mask


def check_attention(got, cache, bits, offs, lens, table, page, q, masks, hq, scale, rows=None):
    hk, d = cache.view.n_kv_heads, cache.view.head_dim
    for b in range(len(offs) - 1):
        m = offs[b + 1] - offs[b]
        if not m:
            continue
        k, v = stored(cache, bits, table, page, b, lens[b] + m)
        mk = oa.chain_masks(m) if masks is None else masks[offs[b]:offs[b + 1]]
        seen = oa.visible(m, lens[b], mk)
        for i in range(m):
            row = offs[b] + i
            if rows is not None and row not in rows:
                continue
            at = np.nonzero(seen[i])[0]
            qi = f64(q[row]).reshape(hq, d)
            for h in range(hq):
                g = f64(got[row]).reshape(hq, d)[h]
                if not len(at):
                    assert np.all(g == 0)
                    continue
                kk, vv = k[at, h // (hq // hk)], v[at, h // (hq // hk)]
                z = scale * (kk @ qi[h])
                p = np.exp(z - z.max())
                p /= p.sum()
                want = p @ vv
                mag = abs(scale) * (np.abs(kk) @ np.abs(qi[h]))
                e = mag * ((2.0 ** -11 if bits != 16 else 0.0) + (d + 8) * U32) + 8 * U32 * (np.abs(z) + np.abs(z).max() + 1)
                rw = (2.0 ** -8 if bits == 16 else 2.0 ** -11) + (np.log2(len(at) + 1) + 16) * U32
                rr = rw + (0.0 if bits == 16 else 2.0 ** -11)
                w = np.expm1(e + rr)                       # a weight's relative change, not to first order only
                den = p @ np.expm1(e + rw)
                assert den < 0.5
                bound = (p @ (np.abs(vv) * w[:, None]) + np.abs(want) * den) / (1 - den)
                bound = bound * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) + 1e-30
                err = np.abs(g - want)
                assert np.all(err <= bound), (b, i, h, float((err / bound).max()))


def tree_masks(r, counts):
    out = []
    for n in counts:
        mine = []
        for i in range(n):
            parent = int(r.integers(0, i)) if i else -1
            mine.append((mine[parent] if i else 0) | 1 << i)
        out += mine
    return out


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("counts,lens,hq,hk,d,page", [
    ([1], [0], 1, 1, 64, 16),                          # one token, nothing before it
    ([1], [1], 4, 1, 128, 16),
    ([1], [127], 4, 2, 128, 16), ([1], [128], 4, 2, 64, 32),          # a tile's last place, and the next tile's first
    ([8], [1000], 8, 2, 128, 64), ([8], [121], 6, 1, 128, 128),
    ([5, 0, 3], [300, 17, 0], 12, 2, 128, 16),         # a request without rows, one without a prefix
    ([17], [95], 5, 1, 64, 256), ([64], [190], 4, 1, 128, 32),         # drafts over two tiles
    ([64, 1], [3, 500], 8, 4, 64, 64), ([33], [65], 6, 1, 128, 16),
    ([2, 7, 1, 20], [513, 40, 2000, 128], 6, 2, 128, 64)])
def test_tree_attention(lib, bits, counts, lens, hq, hk, d, page):
    r = np.random.default_rng(sum(lens) + bits + d)
    for masks in (None, tree_masks(r, counts)):
        cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, hk, d, page, masks)
        scale = d ** -0.5 if masks is None else 0.17
        out = torch.full((offs[-1] + 1, hq * d + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, scale=scale, tree_mask=mask, out=out)
        assert lib.device_error() == 0
        assert torch.all(out[offs[-1]:] == 5.0) and torch.all(out[:, hq * d:] == 5.0)
        check_attention(out[:, :hq * d], cache, bits, offs, lens, table, page, q, masks, hq, scale)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_long_context(lib, bits):
    """Many tiles split over the GPU and joined; the largest scores in one far tile, and spread evenly."""
    r = np.random.default_rng(40 + bits)
    for qscale in (0.2, 6.0):
        counts, lens, hq, hk, d, page = [4, 2], [20011, 7000], 8, 2, 128, 64
        masks = tree_masks(r, counts)
        cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, hk, d, page, masks, qscale=qscale)
        out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, tree_mask=mask)
        check_attention(out, cache, bits, offs, lens, table, page, q, masks, hq, d ** -0.5)
        again = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, tree_mask=mask)
        assert torch.equal(out, again)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("hq,hk", [(4, 1), (16, 1), (24, 1), (64, 1)])
def test_wide_groups(lib, bits, hq, hk):
    r = np.random.default_rng(50 + hq)
    counts, lens = [9, 3], [200, 131]
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, hk, 128, 32)
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq)
    check_attention(out, cache, bits, offs, lens, table, 32, q, None, hq, 128 ** -0.5)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_rows_that_see_nothing_are_zero(lib, bits):
    r = np.random.default_rng(60)
    counts, lens = [4, 3], [0, 0]
    masks = [0b0000, 0b0010, 0b0100, 0, 0, 1 << 40, 0b101]                    # bits past the request's rows do not count
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, 4, 2, 64, 16, masks)
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 4, tree_mask=mask)
    check_attention(out, cache, bits, offs, lens, table, 16, q, [w & 15 for w in masks[:4]] + [w & 7 for w in masks[4:]], 4,
                    64 ** -0.5)
    for row in (0, 3, 4, 5):
        assert torch.all(out[row] == 0)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("length", [0, 5, 125, 300])
def test_what_a_row_does_not_see_stays_out(lib, bits, length):
    """NaN and infinities in drafted keys and values reach the rows that see them and no others."""
    r = np.random.default_rng(70 + length)
    counts, lens = [6], [length]
    masks = [0b000001, 0b000010, 0b000101, 0b001001, 0b010010, 0b110010]
    bad = [float("nan"), float("inf")]

    def spoil(k, v, roff):
        k[length + 2, 5] = bad[0]           # row 2 sees itself
        v[length + 3, 70] = bad[0]          # row 3 sees itself
        v[length + 4, 3] = bad[1]           # rows 4 and 5 see it
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, 4, 2, 128, 16, masks, spoil=spoil)
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 4, tree_mask=mask)
    check_attention(out, cache, bits, offs, lens, table, 16, q, masks, 4, 128 ** -0.5, rows=[0, 1])
    o = f64(out).reshape(6, 4, 128)
    assert np.isnan(o[2, :2]).all() and np.isfinite(o[2, 2:]).all()           # the key's head, every element
    group = slice(64, 128) if bits != 16 else slice(70, 71)                   # a NaN takes its quantized group along
    assert np.isnan(o[3, :2, group]).all() and np.isfinite(o[3, 2:]).all() and np.isfinite(o[3, :2, :64]).all()
    if bits == 16:
        assert np.isposinf(o[4:, :2, 3]).all()
    keep = np.ones(128, bool)
    keep[3] = False
    assert np.isfinite(o[4:, :, keep]).all()


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_extreme_scores(lib, bits):
    """Queries far up and down bf16's range, equal scores, and scores that one token wins."""
    r = np.random.default_rng(80)
    counts, lens = [3], [150]
    for qscale, scale in ((1e30, 2e-31), (1e-30, 2e29), (1e-30, 0.1), (40.0, 128 ** -0.5)):
        cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, 2, 1, 128, 16, qscale=qscale)
        out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 2, scale=scale)
        assert out.isfinite().all()
        check_attention(out, cache, bits, offs, lens, table, 16, q, None, 2, scale)


def test_negative_and_zero_scale(lib):
    r = np.random.default_rng(81)
    counts, lens = [3], [40]
    cache, offs, table, q, mask = attend_case(lib, r, 8, counts, lens, 2, 1, 64, 16)
    for scale in (0.0, -0.3):
        out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 2, scale=scale)
        check_attention(out, cache, 8, offs, lens, table, 16, q, None, 2, scale)


def test_bad_input_is_flagged_by_attention(lib):
    r = np.random.default_rng(82)
    counts, lens = [2, 2], [30, 30]
    cache, offs, table, q, mask = attend_case(lib, r, 16, counts, lens, 2, 1, 64, 16)
    want = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 2)
    lib.device_error()
    for bad_lens, edit in [([30, -3], None), ([30, 10 ** 9], None), ([30, 30], 77), ([30, 30], -1)]:
        t = table.copy()
        if edit is not None:
            t[1, 0] = edit
        out = lib.tree_attention(cache, offs, i32(bad_lens), i32(t.tolist()), q.cuda(), 2)
        assert lib.device_error() == 4
        assert torch.equal(out[:2], want[:2])                                 # the sound request is served
    assert lib.device_error() == 0


def test_binding_refuses(lib):
    r = np.random.default_rng(83)
    cache, offs, table, q, mask = attend_case(lib, r, 16, [2], [30], 2, 1, 64, 16)
    t, n, q = i32(table.tolist()), i32([30]), q.cuda()
    for args in [(n.long(), t, q), (n, t.long(), q), (n, t[0], q), (n, t, q.float()), (n, t, q.cpu()), (n, t, q[:1]),
                 (n, t, q[:, :64])]:
        with pytest.raises(SVError):
            lib.tree_attention(cache, offs, *args, 2)
    with pytest.raises(SVError):
        lib.tree_attention(cache, offs, n, t, q, 2, tree_mask=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(SVError):
        lib.kv_append(cache, offs, n, t, q, q.float())
    with pytest.raises(SVError):
        lib.kv_cache(torch.zeros(2, 1, 16, 64, device="cuda"), torch.zeros(2, 1, 16, 64, device="cuda"))
    with pytest.raises(SVError):
        lib.tree_attention(cache, offs, n, t, q, 2, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------- streams, graphs, a round

def test_another_stream_and_a_replayed_graph(lib):
    """The calls follow their stream; a captured round reads kv_len, table and rows anew at each replay."""
    r = np.random.default_rng(90)
    hq, hk, d, page, m = 8, 2, 128, 16, 5
    table, n_pages = tables(r, [400], page)
    t, lens = i32(table.tolist()), i32([0])
    inv = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    base = torch.arange(m, dtype=torch.int32, device="cuda")
    pos = base.clone()
    x = torch.zeros((m, (hq + 2 * hk) * d), dtype=torch.bfloat16, device="cuda")
    out, qr, kr = (torch.zeros((m, n * d), dtype=torch.bfloat16, device="cuda") for n in (hq, hq, hk))

    def step(cache, ws, stream=None):
        lib.qk_norm_rope(x[:, :hq * d], x[:, hq * d:(hq + hk) * d], d, pos, inv, q_out=qr, k_out=kr, stream=stream)
        lib.kv_append(cache, [0, m], lens, t, kr, x[:, (hq + hk) * d:], stream=stream)
        lib.tree_attention(cache, [0, m], lens, t, qr, hq, out=out, workspace=ws, stream=stream)

    caches = [lib.kv_cache_alloc(n_pages, page, hk, d, 8) for _ in range(3)]
    ws = lib.workspace(lib.tree_attention_workspace_bytes(caches[0], [0, m], hq))
    step(caches[2], ws)                                                       # first use outside the capture
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step(caches[0], ws)
    for i in range(40):
        x.copy_(bf16(r, *x.shape))
        lens.fill_(i * m)
        pos.copy_(base + i * m)
        g.replay()
        got = out.clone()
        if i % 2:
            step(caches[1], ws)
        else:
            torch.cuda.synchronize()
            step(caches[1], None, stream=side)
            side.synchronize()
        assert torch.equal(got, out)
    assert all(torch.equal(a, b) for a, b in zip(caches[0].tensors, caches[1].tensors))
    assert lib.device_error() == 0


def test_a_round_with_attention(lib):
    """q|k|v projection -> norm and rotation -> cache -> tree attention -> o projection with residual, then the
    accepted branch is committed: the next round over the committed cache equals one over a cache that only ever
    held the accepted rows."""
    from tests._util import dev_weight
    import synthetic
    r = synthetic.rng(91)
    hidden, hq, hk, d, page = 1024, 8, 2, 128, 16
    wqkv = dev_weight(synthetic.quant_weight(r, (hq + 2 * hk) * d, hidden, 8, synthetic.LARGE_8BIT))
    wo = dev_weight(synthetic.quant_weight(r, hidden, hq * d, 8, synthetic.LARGE_8BIT))
    inv = torch.from_numpy((1e4 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()
    qw, kw = (1 + bf16(r, d, scale=0.1)).cuda(), (1 + bf16(r, d, scale=0.1)).cuda()

    def layer(cache, table, h, length, depth, masks):
        m = h.shape[0]
        ws = lib.workspace(max(lib.qmm_workspace_bytes(m, (hq + 2 * hk) * d, hidden, 8),
                               lib.qmm_workspace_bytes(m, hidden, hq * d, 8)))
        lib.qmm_prepare(h, hidden, 8, mode=1, workspace=ws)
        qkv = lib.qmm_run(wqkv["wq"], wqkv["scales"], wqkv["biases"], hidden, 8, m, workspace=ws)
        q, k, v = qkv.split([hq * d, hk * d, hk * d], dim=1)
        lib.qk_norm_rope(q, k, d, i32([length + n for n in depth]), inv, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
        lib.kv_append(cache, [0, m], i32([length]), table, k, v)
        mask = None if masks is None else torch.tensor(masks, dtype=torch.int64, device="cuda")
        a = lib.tree_attention(cache, [0, m], i32([length]), table, q, hq, tree_mask=mask)
        aws = lib.workspace(lib.qmm_workspace_bytes(m, hidden, hq * d, 8))
        return lib.qmm_verify(wo["wq"], wo["scales"], wo["biases"], hq * d, 8, a, residual=h, workspace=aws)

    tb = i32(tables(np.random.default_rng(92), [200], page)[0].tolist())
    for bits in (16, 8):
        tree, chain = lib.kv_cache_alloc(20, page, hk, d, bits), lib.kv_cache_alloc(20, page, hk, d, bits)
        prompt = bf16(r, 29, hidden).cuda()
        for c in (tree, chain):
            layer(c, tb, prompt, 0, list(range(29)), None)
        # 0 - 1 - 3 - 5, 0 - 2 - 4: the branch 0, 2, 4 is accepted
        h = bf16(r, 6, hidden).cuda()
        yt = layer(tree, tb, h, 29, [0, 1, 1, 2, 2, 3], [0b1, 0b11, 0b101, 0b1011, 0b10101, 0b101011])
        yc = layer(chain, tb, h[[0, 2, 4]].contiguous(), 29, [0, 1, 2], None)
        lib.kv_commit([tree], i32([29]), tb, i32([[0, 2, 4]]), i32([3]))
        # the same rows through blocks of 6 and 3 rows: equal up to the projections' tile order
        scale = yc.float().abs().max()
        assert (yt[[0, 2, 4]].float() - yc.float()).abs().max() <= 2.0 ** -6 * scale
        kt, vt = lib.kv_read(tree, [0, 32], i32([0]), tb)
        kc, vc = lib.kv_read(chain, [0, 32], i32([0]), tb)
        assert (kt.float() - kc.float()).abs().max() <= 2.0 ** -6 * kc.float().abs().max()
        assert (vt.float() - vc.float()).abs().max() <= 2.0 ** -6 * vc.float().abs().max()
        nxt = bf16(r, 1, hidden).cuda()
        a, b = (layer(c, tb, nxt, 32, [0], None) for c in (tree, chain))
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()
    assert lib.device_error() == 0


# ------------------------------------------------- long calls, and every way that work is split

def rising(k, hk, d, z0=0.0):
    """Scores that climb by up to 20 within a few tiles and fall again, through element 0 of each key (q there is 8, scale 1 / 8)."""
    t = np.arange(len(k))
    level = -60.0 + 20.0 * ((t // 16) % 7) + 12.0 * ((t // 128) % 5) + z0
    k.view(len(k), hk, d)[:, :, 0] = torch.from_numpy(level.astype(np.float32)).to(torch.bfloat16)[:, None]


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("counts,lens,hq,hk,page", [
    ([4], [30003], 8, 2, 64), ([8], [30003], 8, 2, 64),                       # one row tile, two
    ([12], [30003], 8, 2, 128), ([25], [30003], 8, 2, 256),                   # up to 64 rows, up to 128
    ([64], [20001], 8, 2, 64), ([40, 3], [14000, 9000], 8, 2, 16)])           # several blocks of rows
def test_growing_scores(lib, bits, counts, lens, hq, hk, page):
    """Every kernel moves its reference maximum, in runs of several tiles and across joined runs."""
    r = np.random.default_rng(100 + counts[0])
    d = 128
    masks = tree_masks(r, counts)

    def spoil(k, v, roff):
        for b in range(len(counts)):
            rising(k[roff[b]:roff[b + 1]], hk, d)
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, hk, d, page, masks, qscale=0.1, spoil=spoil)
    q.view(offs[-1], hq, d)[:, :, 0] = 8.0
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, scale=0.125, tree_mask=mask)
    assert lib.device_error() == 0
    rows = {0, offs[-1] - 1, offs[1] - 1, offs[1] // 2}
    check_attention(out, cache, bits, offs, lens, table, page, q, masks, hq, 0.125, rows=rows)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("batch,rows,hq", [(3, 4, 8), (24, 9, 8), (48, 5, 16), (96, 4, 8)])
def test_many_requests(lib, bits, batch, rows, hq):
    """Ragged batches whose output rows are joined one to a CTA, eight, and sixteen."""
    r = np.random.default_rng(110 + batch)
    counts = [int(x) for x in r.integers(0, rows + 1, batch)]
    counts[0], counts[-1], counts[1] = rows, 0, 1
    lens = [int(x) for x in r.integers(0, 1500, batch)]
    lens[2] = 4000
    masks = tree_masks(r, counts)
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, 2, 64, 16, masks)
    out = torch.full((offs[-1] + 3, hq * 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, tree_mask=mask, out=out)
    assert lib.device_error() == 0 and torch.all(out[offs[-1]:] == 5.0)
    check_attention(out, cache, bits, offs, lens, table, 16, q, masks, hq, 0.125, rows=set(range(0, offs[-1], 5)))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("counts,lens", [([1, 64, 0, 17, 5], [900, 300, 7, 0, 2000]), ([0, 1, 5, 0, 8], [3, 700, 0, 9, 1300]),
                                         ([5, 1, 1, 0, 0], [100, 300, 0, 0, 0]), ([0, 0, 0, 2, 0], [5, 0, 9, 128, 1])])
def test_mixed_row_counts(lib, bits, counts, lens):
    r = np.random.default_rng(120 + sum(counts))
    masks = tree_masks(r, counts)
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, 8, 2, 128, 32, masks)
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), 8, tree_mask=mask)
    check_attention(out, cache, bits, offs, lens, table, 32, q, masks, 8, 128 ** -0.5)
    none = lib.tree_attention(cache, [0] * 6, i32(lens), i32(table.tolist()), q.cuda(), 8, out=out.clone())
    assert torch.equal(none, out)                                             # no rows: nothing is written


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("m", [3, 14, 40])
def test_empty_masks_in_every_kernel(lib, bits, m):
    """Rows that see nothing are zero beside rows that see something, for any number of rows."""
    r = np.random.default_rng(130 + m)
    masks = [0 if i % 3 == 0 else 1 << i for i in range(m)]
    cache, offs, table, q, mask = attend_case(lib, r, bits, [m], [0], 8, 2, 128, 16, masks)
    out = lib.tree_attention(cache, offs, i32([0]), i32(table.tolist()), q.cuda(), 8, tree_mask=mask)
    check_attention(out, cache, bits, offs, [0], table, 16, q, masks, 8, 128 ** -0.5)
    assert torch.all(out[::3] == 0)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("m,length", [(2, 400), (16, 260), (33, 95)])
def test_strided_rows_and_a_full_table(lib, bits, m, length):
    """q inside a projection's output, out inside a wider buffer and over q; every place of the table in use."""
    r = np.random.default_rng(140 + m)
    hq, hk, d, page = 8, 2, 128, 32
    length = (length + m + page - 1) // page * page - m
    cache, offs, table, q, _ = attend_case(lib, r, bits, [m], [length], hq, hk, d, page)
    t = i32(table[:, :(length + m) // page].tolist())
    want = lib.tree_attention(cache, offs, i32([length]), t, q.cuda(), hq)
    assert lib.device_error() == 0
    check_attention(want, cache, bits, offs, [length], table, page, q, None, hq, d ** -0.5, rows={0, m - 1})
    qkv = torch.full((m + 1, (hq + 4) * d), 3.0, dtype=torch.bfloat16, device="cuda")
    qkv[:m, d:d + hq * d] = q.cuda()
    view = qkv[:m, d:d + hq * d]
    wide = torch.full((m + 1, hq * d + 64), 4.0, dtype=torch.bfloat16, device="cuda")
    lib.tree_attention(cache, offs, i32([length]), t, view, hq, out=wide[:m, 64:])
    assert torch.equal(wide[:m, 64:], want) and torch.all(wide[m:] == 4.0) and torch.all(wide[:, :64] == 4.0)
    lib.tree_attention(cache, offs, i32([length]), t, view, hq, out=view)
    assert torch.equal(view, want)
    assert torch.all(qkv[:, :d] == 3.0) and torch.all(qkv[:, d + hq * d:] == 3.0) and torch.all(qkv[m:] == 3.0)


def test_graphs_that_share_a_workspace(lib):
    """Two captured calls with one workspace, replayed one after the other in any order, and between eager calls."""
    r = np.random.default_rng(150)
    hq, hk, d, page = 8, 2, 128, 16
    calls = []
    for counts, lens, bits in (([3], [3000], 8), ([30, 2], [2000, 700], 16)):
        cache, offs, table, q, _ = attend_case(lib, r, bits, counts, lens, hq, hk, d, page)
        calls.append((cache, lib.row_offsets(offs), i32(lens), i32(table.tolist()), q.cuda(), hq))
    ws = lib.workspace(max(lib.tree_attention_workspace_bytes(c[0], c[1], hq) for c in calls))
    assert not ws.any()
    for c in calls:                                                           # other calls share it and want zeros
        lib.tree_attention(*c, workspace=ws)
        assert not ws.any()
    outs = [torch.zeros_like(c[4]) for c in calls]
    want = [lib.tree_attention(*c) for c in calls]
    graphs = []
    for c, o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            lib.tree_attention(*c, out=o, workspace=ws)
        graphs.append(g)
    for i in (0, 1, 1, 0, 0, 1):
        ws.fill_(255)                                                         # a word read before it is written would be NaN
        outs[i].zero_()
        graphs[i].replay()
        graphs[1 - i].replay()
        assert torch.equal(outs[i], want[i]) and torch.equal(outs[1 - i], want[1 - i])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("counts,hk,d,page", [([700, 1, 333], 8, 128, 64), ([9000, 2001], 1, 64, 16), ([500, 900], 3, 192, 32),
                                              ([40, 220], 16, 256, 16), ([301, 240], 5, 256, 32), ([7, 0, 12], 5, 256, 16)])
def test_long_appends_round_every_tie(lib, bits, counts, hk, d, page):
    """Groups of every magnitude, with half steps that lie exactly between two codes: codes, scales and biases to the last bit."""
    r = np.random.default_rng(160 + d)
    rows = sum(counts)
    top = 2 ** bits - 1
    x = r.integers(0, 2 * top + 1, (rows, hk, d // 64, 64)) / 2.0             # scale 1: every second value is a tie
    x[..., 0], x[..., 1] = 0, top
    e = r.integers(-30, 9, (rows, hk, d // 64, 1)).astype(np.float64)
    x *= 2.0 ** e                                                             # subnormal fp16 scales among them
    x[::7] = r.standard_normal(x[::7].shape) * 2.0 ** r.integers(-4, 5, x[::7].shape)
    k = torch.from_numpy(x.reshape(rows, hk * d).astype(np.float32)).to(torch.bfloat16)
    v = bf16(r, rows, hk * d)
    v.view(-1)[r.integers(0, v.numel(), 50)] = float("inf")
    v.view(-1)[r.integers(0, v.numel(), 50)] = -float("inf")
    v.view(-1)[r.integers(0, v.numel(), 50)] = float("nan")
    lens = [5] * len(counts)
    table, n_pages = tables(r, [n + c for n, c in zip(lens, counts)], page)
    cache = lib.kv_cache_alloc(n_pages, page, hk, d, bits)
    offs = offsets(counts)
    lib.kv_append(cache, offs, i32(lens), i32(table.tolist()), k.cuda(), v.cuda())
    assert lib.device_error() == 0
    got = [t.cpu().numpy() for t in cache.tensors]
    for b, n in enumerate(counts):
        pos = lens[b] + np.arange(n)
        pages, at = table[b, pos // page], pos % page
        for i, rowset in ((0, k), (1, v)):
            c, s, z = oa.kv_quantize(rowset[offs[b]:offs[b + 1]].float().numpy().reshape(n, hk, d), bits)
            assert np.array_equal(got[i][pages, :, at].view(np.uint32), oa.pack(c, bits))
            assert np.array_equal(got[2 + 2 * i][pages, :, at], s, equal_nan=True)
            assert np.array_equal(got[3 + 2 * i][pages, :, at], z, equal_nan=True)
    kk, vv = lib.kv_read(cache, offs, i32(lens), i32(table.tolist()))
    short = [torch.cat(p) for p in zip(*[lib.kv_read(cache, [0, 100], i32([lens[0] + a]), i32(table[:1].tolist()))
                                         for a in range(0, counts[0] - 99, 100)])]
    for long, part in zip((kk, vv), short):                                   # the long call's values are the short calls'
        a, b = long[:len(part)].view(torch.int16), part.view(torch.int16)
        assert torch.equal(a, b) and len(part) == counts[0] // 100 * 100


@pytest.mark.parametrize("rows,hq,hk,d,rot,interleaved,norm", [
    (801, 48, 8, 128, 64, True, True), (2500, 12, 3, 128, 128, False, True), (3300, 18, 2, 64, 32, False, False),
    (2000, 9, 2, 80, 80, True, True), (700, 40, 7, 256, 128, False, True), (1200, 33, 1, 128, 0, False, True)])
def test_norm_rope_of_prompts(lib, rows, hq, hk, d, rot, interleaved, norm):
    r = np.random.default_rng(170 + d)
    q, k = bf16(r, rows, hq * d, scale=3.0).cuda(), bf16(r, rows, hk * d).cuda()
    qw, kw = (1 + bf16(r, d, scale=0.2)).cuda(), (1 + bf16(r, d, scale=0.2)).cuda()
    pos = r.integers(0, 1000000, rows)
    inv = (1e6 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    args = dict(positions=i32(pos.tolist()), inv_freq=torch.from_numpy(inv).cuda()) if rot else {}
    qo, ko = lib.qk_norm_rope(q, k, d, q_weight=qw, k_weight=kw, norm=norm, interleaved=interleaved, **args)
    some = sorted(set(range(0, rows, 13)) | {rows - 1})
    for out, x, w, n in ((qo, q, qw, hq), (ko, k, kw, hk)):
        check_rope(f64(out[some]).reshape(-1, n, d), f64(x[some]).reshape(-1, n, d), f64(w), norm, pos[some], inv if rot else None,
                   interleaved)
    one, _ = lib.qk_norm_rope(q[7:8], None, d, q_weight=qw, norm=norm, interleaved=interleaved,
                              **(dict(args, positions=args["positions"][7:8]) if rot else {}))
    assert torch.equal(one[0], qo[7])                                         # few rows and many: the same values


def test_rope_at_the_ends_of_the_positions(lib):
    """Angles are exact products mod a turn: any int32 position, frequencies from 2^-40 to 2^23 (of either sign); from 2^24 on
    and for infinity and NaN the pair is NaN."""
    r = np.random.default_rng(180)
    d, e = 64, [0, -1, 3, -7, -40, -20, 10, 23, -31, 1, 5, -3, 2, -10, -15, 7]
    inv = np.array([2.0 ** x * (-1 if i % 3 == 2 else 1) for i, x in enumerate(e)] +
                   [2.0 ** 24, 3e38, -2.0 ** 30, np.inf, -np.inf, np.nan, 0.0, 2.0 ** -149] + [1.0] * 8, np.float32)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -7654321, 65536]
    x = bf16(r, len(pos), d).cuda()
    got, _ = lib.qk_norm_rope(x, None, d, i32(pos), torch.from_numpy(inv).cuda(), norm=False)
    good = np.isfinite(inv) & (np.abs(inv) < 2.0 ** 24)
    g, xs = f64(got), f64(x)
    assert np.isnan(g[:, :32][:, ~good]).all() and np.isnan(g[:, 32:][:, ~good]).all()
    # positions times powers of two are exact in fp64, and the C library reduces them mod 2 pi exactly
    a = np.array(pos, np.float64)[:, None] * np.where(good, inv, 0).astype(np.float64)
    c, s = np.vectorize(math.cos)(a), np.vectorize(math.sin)(a)
    want = np.concatenate([xs[:, :32] * c - xs[:, 32:] * s, xs[:, 32:] * c + xs[:, :32] * s], 1)
    keep = np.concatenate([good, good])
    pair = np.abs(xs[:, :32]) + np.abs(xs[:, 32:])
    bound = 2.0 ** -8 * np.abs(want) + 32 * U32 * np.concatenate([pair, pair], 1) + 1e-38
    assert np.all(np.abs(g - want)[:, keep] <= bound[:, keep])


@pytest.mark.parametrize("bits", [16, 8])
def test_a_cache_past_32_bits(lib, bits):
    """Pages beyond 2^31 elements (and, in 16 bits, 2^32 bytes): the calls give what they give in a small cache."""
    r = np.random.default_rng(190)
    hk, d, page, hq = 8, 128, 256, 16
    n_pages = 2 ** 31 // (hk * d * page) + 9
    big, small = lib.kv_cache_alloc(n_pages, page, hk, d, bits), lib.kv_cache_alloc(9, page, hk, d, bits)
    at = [n_pages - 9 + i for i in (4, 0, 8, 2)], [4, 0, 8, 2]
    rows = bf16(r, 1000, 2 * hk * d).cuda()
    for m in (2, 20, 64):
        q = bf16(r, m, hq * d).cuda()
        got = []
        for cache, pages in zip((big, small), at):
            t = i32([pages])
            lib.kv_append(cache, [0, 1000], i32([0]), t, rows[:, :hk * d], rows[:, hk * d:])
            o = lib.tree_attention(cache, [0, m], i32([1000 - m]), t, q, hq)
            lib.kv_commit([cache], i32([1000 - m]), t, i32([[1] if m == 2 else [1, 5, 19]]), i32([1 if m == 2 else 3]))
            got.append([o] + list(lib.kv_read(cache, [0, 1000], i32([0]), t)))
        assert lib.device_error() == 0
        assert all(torch.equal(a, b) for a, b in zip(*got))
        assert got[0][0].float().abs().max() > 0


def test_commit_refuses_a_cache_listed_twice(lib):
    cache, other = (lib.kv_cache_alloc(2, 16, 1, 64, 16) for _ in range(2))
    args = (i32([0]), i32([[0, 1]]), i32([[2]]), i32([1]))
    lib.kv_commit([cache, other], *args)
    with pytest.raises(SVError):
        lib.kv_commit([cache, other, cache], *args)
    with pytest.raises(SVError):
        lib.kv_append(lib.kv_cache(cache.k, cache.k), [0, 1], i32([0]), i32([[0, 1]]), other.k[0, 0, :1], other.k[0, 0, :1])


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("hq", [16, 32, 64])                                  # 48, 96 and 192 rows a key head
@pytest.mark.parametrize("length", [0, 125, 2500])
def test_what_a_row_does_not_see_stays_out_of_wide_blocks(lib, bits, hq, length):
    r = np.random.default_rng(200 + length + hq)
    masks = [0b000001, 0b000010, 0b000101, 0b001001, 0b010010, 0b110010]

    def spoil(k, v, roff):
        k[length + 2, 5] = float("nan")
        v[length + 3, 70] = float("nan")
        v[length + 4, 3] = float("inf")
    cache, offs, table, q, mask = attend_case(lib, r, bits, [6], [length], hq, 2, 128, 16, masks, spoil=spoil)
    out = lib.tree_attention(cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq, tree_mask=mask)
    check_attention(out, cache, bits, offs, [length], table, 16, q, masks, hq, 128 ** -0.5, rows=[0, 1])
    o, half = f64(out).reshape(6, hq, 128), hq // 2
    assert np.isnan(o[2, :half]).all() and np.isfinite(o[2, half:]).all()
    group = slice(64, 128) if bits != 16 else slice(70, 71)
    assert np.isnan(o[3, :half, group]).all() and np.isfinite(o[3, half:]).all() and np.isfinite(o[3, :half, :64]).all()
    if bits == 16:
        assert np.isposinf(o[4:, :half, 3]).all()
    keep = np.ones(128, bool)
    keep[3] = False
    assert np.isfinite(o[4:, :, keep]).all()


def test_binding_refuses_what_is_missing(lib):
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(SVError):
        lib.qk_norm_rope(x, None, 64, None, torch.ones(32, device="cuda"))    # an angle without a position
    cache = lib.kv_cache_alloc(2, 16, 1, 64, 16)
    for offs in ([0], [0, 3, 1], [1, 2], [0, -1]):
        with pytest.raises(SVError):
            lib.kv_append(cache, offs, i32([0, 0]), i32([[0, 1], [1, 0]]), x, x)
        with pytest.raises(SVError):
            lib.tree_attention(cache, offs, i32([0, 0]), i32([[0, 1], [1, 0]]), x, 1)


def test_results_on_a_side_stream_do_not_share_memory_with_pending_work(lib):
    """What a call on another stream allocates is not memory that the current stream still works on."""
    r = np.random.default_rng(210)
    counts, lens = [3], [300]
    cache, offs, table, q, _ = attend_case(lib, r, 16, counts, lens, 8, 2, 64, 16)
    q, n, t = q.cuda(), i32(lens), i32(table.tolist())
    want = lib.tree_attention(cache, offs, n, t, q, 8)
    side, big = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        y = big
        for _ in range(20):
            y = y @ big                                                       # pending on the current stream
        scratch = torch.zeros_like(want)
        scratch += y[0, 0].to(torch.bfloat16)                                 # written after all of it
        del scratch                                                           # and free for the current stream's next tensor
        got = lib.tree_attention(cache, offs, n, t, q, 8, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [16, 8])
def test_the_largest_batch_and_the_widest_request(lib, bits):
    r = np.random.default_rng(220 + bits)
    counts, lens = [int(x) for x in r.integers(0, 3, 256)], [int(x) for x in r.integers(0, 200, 256)]
    counts[255] = 2
    masks = tree_masks(r, counts)
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, 2, 1, 64, 16, masks)
    n = i32([a if c else -7 for a, c in zip(lens, counts)])                   # lengths of requests without rows are not looked at
    out = lib.tree_attention(cache, offs, n, i32(table.tolist()), q.cuda(), 2, tree_mask=mask)
    assert lib.device_error() == 0
    check_attention(out, cache, bits, offs, lens, table, 16, q, masks, 2, 0.125)
    path = np.zeros((256, 1), dtype=np.int32)
    path[255, 0] = 1
    before = lib.kv_read(cache, [0] * 256 + [1], i32([0] * 255 + [lens[255] + 1]), i32(table.tolist()))
    lib.kv_commit([cache], n, i32(table.tolist()), i32(path.tolist()), i32([0] * 255 + [1]))
    after = lib.kv_read(cache, [0] * 256 + [1], i32([0] * 255 + [lens[255]]), i32(table.tolist()))
    assert lib.device_error() == 0 and all(torch.equal(a, b) for a, b in zip(before, after))

    counts, lens, hq = [64], [140], 64                                        # 4096 rows over one key head
    masks = tree_masks(r, counts)
    cache, offs, table, q, mask = attend_case(lib, r, bits, counts, lens, hq, 1, 128, 64, masks)
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, tree_mask=mask)
    assert lib.device_error() == 0
    check_attention(out, cache, bits, offs, lens, table, 64, q, masks, hq, 128 ** -0.5, rows={0, 1, 31, 32, 62, 63})


def test_two_streams_at_once(lib):
    """Rounds on two streams, each with its own cache and workspace, do not touch each other."""
    r = np.random.default_rng(230)
    hq, hk, d, page = 8, 2, 128, 32
    sides = []
    for counts, lens, bits in (([7, 2], [3000, 500], 8), ([40], [2500], 16)):
        cache, offs, table, q, _ = attend_case(lib, r, bits, counts, lens, hq, hk, d, page)
        offs = lib.row_offsets(offs)
        rows = [bf16(r, offs[len(counts)], hk * d).cuda() for _ in range(2)]
        args = (cache, offs, i32(lens), i32(table.tolist()))
        ws = lib.workspace(lib.tree_attention_workspace_bytes(cache, offs, hq))
        lib.kv_append(*args, *rows)
        want = lib.tree_attention(*args, q.cuda(), hq)
        path = i32([[1, 2]] * len(counts)), i32([2] + [0] * (len(counts) - 1))
        sides.append((args, rows, q.cuda(), ws, want, path, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        for args, rows, q, ws, want, path, stream in sides:
            with torch.cuda.stream(stream):
                lib.kv_append(*args, *rows)
                outs.append((lib.tree_attention(*args, q, hq, workspace=ws), want))
                lib.kv_commit([args[0]], args[2], args[3], *path)             # undone by the next append
    torch.cuda.synchronize()
    assert lib.device_error() == 0 and all(torch.equal(a, b) for a, b in outs)
