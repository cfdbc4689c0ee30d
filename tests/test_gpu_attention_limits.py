"""Tree attention where its number formats end: references that move in every chunk of tokens, far queries and values,
weights at the bottom of fp16, codes at the top of it.

The tolerance is that of test_gpu_attention.py (its docstring derives it) and one term more.  Over codes a weight is fp16,
and below 2^-14 its rounding is no longer relative: it is off by up to 2^-25.  A row's reference is set so that its largest
weight then is 2^5, and stays there or grows; so that is at most 2^-30 of the largest weight, and a token's share of
the numerator moves by up to 2^-30 max(p) |v|.  A run of a row with a lower maximum of its own is nearer still.  Over a 16-bit
cache weights are bf16, whose range is fp32's: nothing is added.
"""

import numpy as np
import pytest
import torch

from speculative_decoding_verify_qmm_gb300.binding import SVError
from tests.test_gpu_attention import U32, attend_case, f64, i32, stored

pytestmark = pytest.mark.gpu


def check(got, cache, bits, offs, lens, table, page, q, hq, scale, requests=None):
    """Every row of chains (of some requests) against fp64."""
    hk, d = cache.view.n_kv_heads, cache.view.head_dim
    tail = 2.0 ** -30 if bits != 16 else 0.0
    worst = 0.0
    for b in requests or range(len(offs) - 1):
        m = offs[b + 1] - offs[b]
        k, v = stored(cache, bits, table, page, b, lens[b] + m)
        for i in range(m):
            n = lens[b] + i + 1
            qi, gi = f64(q[offs[b] + i]).reshape(hq, d), f64(got[offs[b] + i]).reshape(hq, d)
            for h in range(hq):
                kk, vv = k[:n, h // (hq // hk)], v[:n, h // (hq // hk)]
                z = scale * (kk @ qi[h])
                p = np.exp(z - z.max())
                p /= p.sum()
                want = p @ vv
                mag = abs(scale) * (np.abs(kk) @ np.abs(qi[h]))
                e = mag * ((2.0 ** -11 if bits != 16 else 0.0) + (d + 8) * U32) + 8 * U32 * (np.abs(z) + np.abs(z).max() + 1)
                rw = (2.0 ** -8 if bits == 16 else 2.0 ** -11) + (np.log2(n + 1) + 16) * U32
                rr = rw + (0.0 if bits == 16 else 2.0 ** -11)
                den = p @ np.expm1(e + rw)
                assert den < 0.5
                bound = ((p * np.expm1(e + rr) + tail * p.max()) @ np.abs(vv) + np.abs(want) * den) / (1 - den)
                bound = bound * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(want) + 1e-30
                worst = max(worst, float((np.abs(gi[h] - want) / bound).max()))
    assert worst <= 1, worst


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("hq", [3, 8, 16, 32])                                # 9, 24, 48 and 96 rows over one key head
@pytest.mark.parametrize("first", [0, 96])
def test_a_reference_that_moves_in_every_chunk(lib, bits, hq, first):
    """Scores climb by 11 (16 powers of two) every 32 tokens of a tile of 128, so the weights that a tile has so far are read
    back and rescaled; the values of the tokens one step below the top are large enough to count."""
    r = np.random.default_rng(300 + hq + first)
    d, m, length = 128, 3, 700 + first
    step = np.arange(length + m) // 32 % 4

    def spoil(k, v, roff):
        k[:, 0] = torch.from_numpy((11.0 * step - 16.0).astype(np.float32)).to(torch.bfloat16)
        v *= torch.from_numpy(np.where(step == 2, 4096.0, 1.0).astype(np.float32)).to(torch.bfloat16)[:, None]
    cache, offs, table, q, _ = attend_case(lib, r, bits, [m], [length], hq, 1, d, 64, qscale=0.05, spoil=spoil)
    q.view(m, hq, d)[:, :, 0] = 8.0
    args = (cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq)
    out = lib.tree_attention(*args, scale=0.125)
    assert lib.device_error() == 0
    check(out, cache, bits, offs, [length], table, 64, q, hq, 0.125)
    for _ in range(20):
        assert torch.equal(lib.tree_attention(*args, scale=0.125), out)


@pytest.mark.parametrize("hq", [3, 8, 16, 32])
@pytest.mark.parametrize("climb,size", [(35.0, 2.0 ** 110), (0.0, 3e38), (35.0, 2.0 ** -90)])
def test_large_and_small_values_of_a_16_bit_cache(lib, hq, climb, size):
    """Finite values give finite averages, however far scores have climbed since the reference was set: by 40 powers of two in each
    SM's share of 128 requests."""
    r = np.random.default_rng(310 + hq)
    d, m, length, batch = 128, 3, 1500, 128

    def spoil(k, v, roff):
        for b in range(batch):
            k[roff[b]:roff[b + 1], 0] = torch.linspace(-climb / 2, climb / 2, length + m).to(torch.bfloat16)
        v.copy_((v.double().clamp(-1, 1) * size).to(torch.bfloat16) if climb else torch.full_like(v, size))
    lens = [length] * batch
    cache, offs, table, q, _ = attend_case(lib, r, 16, [m] * batch, lens, hq, 1, d, 64, qscale=0.05, spoil=spoil)
    q.view(m * batch, hq, d)[:, :, 0] = 8.0
    out = lib.tree_attention(cache, offs, i32(lens), i32(table.tolist()), q.cuda(), hq, scale=0.125)
    assert lib.device_error() == 0 and out.isfinite().all()
    check(out, cache, 16, offs, lens, table, 64, q, hq, 0.125, requests=range(0, batch, 41))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq", [3, 8, 16, 32])
@pytest.mark.parametrize("size,scale", [(3e37, 2e-38), (2.0 ** 117, 2.0 ** -117), (2.0 ** -125, 2.0 ** 124), (2.0 ** -131, 2.0 ** 127)])
def test_queries_of_any_size_over_codes(lib, bits, hq, size, scale):
    """A row of q enters the products as fp16 times a power of two, for any finite bf16 values."""
    r = np.random.default_rng(320 + hq)
    d, m, length = 128, 3, 300
    cache, offs, table, q, _ = attend_case(lib, r, bits, [m], [length], hq, 1, d, 64, qscale=1.0)
    q = (q.double() * size / 3).to(torch.bfloat16)
    assert q.isfinite().all()
    out = lib.tree_attention(cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq, scale=scale)
    assert lib.device_error() == 0 and out.isfinite().all()
    check(out, cache, bits, offs, [length], table, 64, q, hq, scale)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("hq", [3, 8, 16, 32])
def test_a_long_tail_behind_large_weights(lib, bits, hq):
    """Every 16th token has a weight 2^22 to 2^30 times the others', and zeros in half of the head: there the output is the tail's alone."""
    r = np.random.default_rng(330 + hq)
    d, m, length = 128, 3, 5000

    def spoil(k, v, roff):
        large = torch.arange(length + m) % 16 == 0
        far = -np.log(2) * r.uniform(22, 30, length + m)
        k[:, 0] = torch.where(large, torch.zeros(length + m), torch.from_numpy(far.astype(np.float32))).to(torch.bfloat16)
        v.abs_()
        v[large, :64] = 0
    cache, offs, table, q, _ = attend_case(lib, r, bits, [m], [length], hq, 1, d, 64, qscale=0.02, spoil=spoil)
    q.view(m, hq, d)[:, :, 0] = 8.0
    out = lib.tree_attention(cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq, scale=0.125)
    assert lib.device_error() == 0
    check(out, cache, bits, offs, [length], table, 64, q, hq, 0.125)
    assert torch.all(out.view(m, hq, d)[:, :, :64] > 0)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("hq", [3, 8, 16, 32])
def test_codes_at_the_top_of_fp16(lib, bits, hq):
    """A cache that the caller filled: scales of either sign, values up to 65504 in magnitude and no further."""
    r = np.random.default_rng(340 + hq)
    d, m, length = 128, 3, 400
    cache, offs, table, q, _ = attend_case(lib, r, bits, [m], [length], hq, 1, d, 64, qscale=2.0 ** -16)
    top = 2 ** bits - 1
    for t in cache.tensors[:2]:
        t.copy_(torch.from_numpy(r.integers(-2 ** 31, 2 ** 31, tuple(t.shape))).to(torch.int32))
    for s, z in (cache.tensors[2:4], cache.tensors[4:6]):
        scale = torch.from_numpy(r.uniform(0, 65504 * 2 / top, tuple(s.shape))).to(torch.float16).double()
        bias = (65504 - scale * top).clamp(-65504, 65504).to(torch.float16).double()
        bias = torch.where(scale * top + bias > 65504, torch.zeros_like(bias), bias)      # (its rounding went up)
        scale = torch.where(scale * top + bias > 65504, torch.zeros_like(scale), scale)
        sign = torch.from_numpy(r.choice([-1.0, 1.0], tuple(s.shape)))
        s.copy_((scale * sign).to(torch.float16))
        z.copy_((bias * sign).to(torch.float16))
    out = lib.tree_attention(cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq, scale=0.125)
    assert lib.device_error() == 0 and out.isfinite().all()
    check(out, cache, bits, offs, [length], table, 64, q, hq, 0.125)


def test_a_workspace_with_gaps_is_refused(lib):
    """The call writes adjacent bytes: between a strided tensor's elements is another's memory."""
    r = np.random.default_rng(350)
    cache, offs, table, q, _ = attend_case(lib, r, 16, [2], [30], 2, 1, 64, 16)
    args = (cache, offs, i32([30]), i32(table.tolist()), q.cuda(), 2)
    n = lib.tree_attention_workspace_bytes(cache, offs, 2)
    with pytest.raises(SVError):
        lib.tree_attention(*args, workspace=torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2])
    assert torch.equal(lib.tree_attention(*args, workspace=lib.workspace(n)), lib.tree_attention(*args))
