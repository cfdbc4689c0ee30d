"""Attention over shared prefixes where its number formats end, as test_gpu_attention_limits.py asks of tree attention: references that move
in every chunk of tokens, far queries and values, weights at the bottom of fp16, codes at the top of it.

Formats and rules are tree attention's, so the tolerance is too (derived there): a part's weights are rounded relative to its own
largest, which is no larger than the row's, and the join adds parts in fp32, inside the (log2 T + 16) u32 of a sum.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_attention_limits import check
from tests.test_gpu_attention_shared import Batch

pytestmark = pytest.mark.gpu

HK, D, PAGE = 8, 128, 64
# drafted rows of a request and query heads per key head: 46, 138, 276 and 414 rows of 46 requests over a key head, so blocks whose two matrices
# take every other tile, the same tiles, and both kinds
ROWS = [(1, 1), (3, 1), (3, 2), (3, 3)]


def batch(lib, seed, bits, m, per, qscale, spoil=None, requests=46, pages=22, own=50):
    b = Batch(lib, seed, bits, [[(m, own + i % 9) for i in range(requests)]], [pages], HK * per, HK, D, PAGE, masks=None, qscale=qscale, spoil=spoil)
    assert b.shares()
    return b


def first_column(b, value):
    b.q.view(-1, b.hq, D)[:, :, 0] = value
    b.q_d = b.q.cuda()


def verify(lib, b, out, scale, requests=(0, 20, 45)):
    assert lib.device_error() == 0 and out.isfinite().all()
    check(out, b.cache, b.bits, b.offs, b.lens, b.table, PAGE, b.q, b.hq, scale, requests=list(requests))


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("m,per", ROWS)
@pytest.mark.parametrize("chunk", [32, 64, 128])
def test_a_reference_that_moves_in_every_chunk(lib, bits, m, per, chunk):
    """Scores climb by 11 (16 powers of two) every 32, 64 or 128 tokens, four times; the values one step below the top are large enough to count."""
    def spoil(k, v, roff, n):
        for i in range(len(roff) - 1):                            # (of the prefix, and of each request's own tokens)
            step = np.arange(roff[i + 1] - roff[i]) // chunk % 4
            k[roff[i]:roff[i + 1]].view(-1, HK, D)[:, :, 0] = torch.from_numpy((11.0 * step - 16.0).astype(np.float32)).to(torch.bfloat16)[:, None]
            v[roff[i]:roff[i + 1]] *= torch.from_numpy(np.where(step == 2, 4096.0, 1.0).astype(np.float32)).to(torch.bfloat16)[:, None]
    b = batch(lib, 400 + chunk + per, bits, m, per, 0.05, spoil)
    first_column(b, 8.0)
    out = b.call(scale=0.125)
    verify(lib, b, out, 0.125)
    for _ in range(10):
        assert torch.equal(b.call(scale=0.125), out)


@pytest.mark.parametrize("m,per", ROWS)
@pytest.mark.parametrize("climb,size", [(35.0, 2.0 ** 110), (-35.0, 2.0 ** 110), (0.0, 3e38), (35.0, 2.0 ** -90)])
def test_large_and_small_values_of_a_16_bit_cache(lib, m, per, climb, size):
    """Finite values give finite averages, however far scores climb or fall over the prefix and the own tokens."""
    def spoil(k, v, roff, n):
        for i in range(len(roff) - 1):
            k[roff[i]:roff[i + 1]].view(-1, HK, D)[:, :, 0] = torch.linspace(-climb / 2, climb / 2, roff[i + 1] - roff[i]).to(torch.bfloat16)[:, None]
        v.copy_((v.double().clamp(-1, 1) * size).to(torch.bfloat16) if climb else torch.full_like(v, size))
    b = batch(lib, 410 + per, 16, m, per, 0.05, spoil)
    first_column(b, 8.0)
    verify(lib, b, b.call(scale=0.125), 0.125)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("m,per", ROWS)
@pytest.mark.parametrize("size,scale", [(3e37, 2e-38), (2.0 ** 117, 2.0 ** -117), (2.0 ** -125, 2.0 ** 124), (2.0 ** -131, 2.0 ** 127)])
def test_queries_of_any_size_over_codes(lib, bits, m, per, size, scale):
    """A row of q enters the products as fp16 times a power of two, for any finite bf16 values."""
    b = batch(lib, 420 + per, bits, m, per, 1.0)
    b.q = (b.q.double() * size / 3).to(torch.bfloat16)
    assert b.q.isfinite().all()
    b.q_d = b.q.cuda()
    verify(lib, b, b.call(scale=scale), scale)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("m,per", ROWS)
@pytest.mark.parametrize("where", ["prefix", "own", "both"])
def test_a_long_tail_behind_large_weights(lib, bits, m, per, where):
    """Every 16th token has a weight 2^22 to 2^30 times the others', and zeros in half of the head: there the output is the tail's alone."""
    r = np.random.default_rng(430 + per)

    def spoil(k, v, roff, n):
        rows = roff[-1]
        large = torch.arange(rows) % 16 == 0
        if where != "both":
            large[slice(roff[n], None) if where == "prefix" else slice(0, roff[n])] = False
        far = torch.from_numpy((-np.log(2) * r.uniform(22, 30, rows)).astype(np.float32))
        k.view(-1, HK, D)[:, :, 0] = torch.where(large, torch.zeros(rows), far).to(torch.bfloat16)[:, None]
        v.abs_()
        v.view(-1, HK, D)[large, :, :64] = 0
    b = batch(lib, 430 + per, bits, m, per, 0.02, spoil)
    first_column(b, 8.0)
    out = b.call(scale=0.125)
    verify(lib, b, out, 0.125)
    assert torch.all(out.view(-1, b.hq, D)[:, :, :64] > 0)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("m,per", ROWS)
def test_codes_at_the_top_of_fp16(lib, bits, m, per):
    """A cache that the caller filled: scales of either sign, values up to 65504 in magnitude and no further."""
    r = np.random.default_rng(440 + per)
    b = batch(lib, 440 + per, bits, m, per, 2.0 ** -16)
    top = 2 ** bits - 1
    for t in b.cache.tensors[:2]:
        t.copy_(torch.from_numpy(r.integers(-2 ** 31, 2 ** 31, tuple(t.shape))).to(torch.int32))
    for s, z in (b.cache.tensors[2:4], b.cache.tensors[4:6]):
        scale = torch.from_numpy(r.uniform(0, 65504 * 2 / top, tuple(s.shape))).to(torch.float16).double()
        bias = (65504 - scale * top).clamp(-65504, 65504).to(torch.float16).double()
        bias = torch.where(scale * top + bias > 65504, torch.zeros_like(bias), bias)      # (its rounding went up)
        scale = torch.where(scale * top + bias > 65504, torch.zeros_like(scale), scale)
        sign = torch.from_numpy(r.choice([-1.0, 1.0], tuple(s.shape)))
        s.copy_((scale * sign).to(torch.float16))
        z.copy_((bias * sign).to(torch.float16))
    verify(lib, b, b.call(scale=0.125), 0.125)
