"""Pins of the attention oracle: closed forms, hand examples and invariants."""

import numpy as np
import pytest

from oracle import attention as oa


def test_rotation_closed_forms():
    r = np.random.default_rng(0)
    x = r.standard_normal((3, 2, 8))
    inv = np.array([0.5, 0.25])
    same = oa.norm_rope(x, None, 0.0, False, [0, 0, 0], inv, False)
    assert np.array_equal(same, x)
    # a quarter turn takes (a, b) to (-b, a), on the pair (p, p + half) or (2p, 2p + 1)
    quarter = np.array([np.pi / 2])
    y = oa.norm_rope(np.array([[[1.0, 2.0, 3.0, 4.0]]]), None, 0.0, False, [1], quarter, True)
    assert np.allclose(y, [[[-2.0, 1.0, 3.0, 4.0]]])
    y = oa.norm_rope(np.array([[[1.0, 2.0, 3.0, 4.0]]]), None, 0.0, False, [1], np.array([np.pi / 2, 0.0]), False)
    assert np.allclose(y, [[[-3.0, 2.0, 1.0, 4.0]]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_products_depend_on_the_distance_alone(interleaved):
    r = np.random.default_rng(1)
    q, k = r.standard_normal((1, 1, 16)), r.standard_normal((1, 1, 16))
    inv = 10.0 ** -np.arange(8.0)
    def dot(a, b):
        return float((oa.norm_rope(q, None, 0, False, [a], inv, interleaved)
                      * oa.norm_rope(k, None, 0, False, [b], inv, interleaved)).sum())
    assert abs(dot(7, 3) - dot(1004, 1000)) < 1e-9
    assert abs(dot(7, 3) - dot(7, 4)) > 1e-6


def test_head_norm():
    x = np.full((1, 1, 4), 3.0)
    y = oa.norm_rope(x, np.array([1.0, 2.0, 3.0, 4.0]), 0.0, True, None, None, False)
    assert np.allclose(y, [[[1.0, 2.0, 3.0, 4.0]]])
    y = oa.norm_rope(x, None, 7.0, True, None, None, False)
    assert np.allclose(y, 3.0 / 4.0)


@pytest.mark.parametrize("bits", [4, 8])
def test_quantizer(bits):
    r = np.random.default_rng(2)
    x = r.standard_normal((5, 128)).astype(np.float32)
    c, s, b = oa.kv_quantize(x, bits)
    y = oa.kv_dequantize(c, s, b)
    # half a step, plus what the scale's and bias's fp16 rounding moves the far end by
    step = np.repeat(s.astype(np.float64), 64, axis=-1)
    assert np.all(np.abs(y - x) <= step * 0.5 + (2 ** bits) * step * 2.0 ** -11 + np.abs(x).max() * 2.0 ** -11)
    assert c.min() == 0 and c.max() >= 2 ** bits - 2
    assert np.array_equal(oa.unpack(oa.pack(c, bits), bits), c)
    # codes that are already on the grid come back exactly
    grid = np.tile(np.arange(64) % (2 ** bits), 1).astype(np.float32)
    grid[0], grid[1] = 0, 2 ** bits - 1
    c, s, b = oa.kv_quantize(grid[None], bits)
    assert s[0, 0] == 1 and b[0, 0] == 0 and np.array_equal(c[0], grid)


def test_quantizer_edges():
    flat = np.full((1, 64), 1.5, dtype=np.float32)
    c, s, b = oa.kv_quantize(flat, 8)
    assert s[0, 0] == 0 and np.all(oa.kv_dequantize(c, s, b) == 1.5)
    far = np.zeros((1, 64), dtype=np.float32)
    far[0, 0], far[0, 1] = np.inf, -3e38
    c, s, b = oa.kv_quantize(far, 8)
    y = oa.kv_dequantize(c, s, b)
    assert np.all(np.isfinite(y)) and np.abs(y).max() < 65504
    nan = np.zeros((1, 128), dtype=np.float32)
    nan[0, 3] = np.nan
    y = oa.kv_dequantize(*oa.kv_quantize(nan, 4))
    assert np.isnan(y[0, :64]).all() and np.all(y[0, 64:] == 0)


def test_words_are_the_weight_format():
    from oracle import quant
    codes = np.random.default_rng(3).integers(0, 16, (2, 64))
    assert np.array_equal(oa.pack(codes, 4), quant.pack_codes(codes, 4))


def test_attention_means_and_picks():
    v = np.arange(12.0).reshape(3, 1, 4)
    k = np.zeros((3, 1, 4))
    q = np.ones((1, 2, 4))
    o = oa.tree_attention(q, k, v, 2, [1], 1.0)
    assert np.allclose(o, v.mean(axis=0))                       # equal scores: the mean
    k[1] = 100.0
    assert np.allclose(oa.tree_attention(q, k, v, 2, [1], 1.0), v[1])   # one dominates
    assert np.allclose(oa.tree_attention(q, k, v, 2, [0], 1.0), v[1])
    assert np.all(oa.tree_attention(q, k[:1], v[:1], 0, [0], 1.0) == 0)  # nothing to see


def test_a_chain_equals_one_token_at_a_time():
    r = np.random.default_rng(4)
    q, k, v = r.standard_normal((4, 4, 8)), r.standard_normal((9, 2, 8)), r.standard_normal((9, 2, 8))
    whole = oa.tree_attention(q, k, v, 5, oa.chain_masks(4), 0.3)
    for i in range(4):
        one = oa.tree_attention(q[i:i + 1], k[:6 + i], v[:6 + i], 5 + i, [1], 0.3)
        assert np.allclose(whole[i], one[0])


def test_a_tree_equals_its_branches():
    """Rows of a two-branch tree see what a chain made of their own branch sees."""
    r = np.random.default_rng(5)
    q, k, v = r.standard_normal((5, 2, 8)), r.standard_normal((8, 2, 8)), r.standard_normal((8, 2, 8))
    masks = [0b1, 0b11, 0b101, 0b1011, 0b10101]               # 0 - 1 - 3 and 0 - 2 - 4
    tree = oa.tree_attention(q, k, v, 3, masks, 1.0)
    for branch in ([0, 1, 3], [0, 2, 4]):
        at = [0, 1, 2] + [3 + j for j in branch]
        chain = oa.tree_attention(q[branch], k[at], v[at], 3, oa.chain_masks(3), 1.0)
        assert np.allclose(tree[branch], chain)


def test_unseen_rows_do_not_matter():
    r = np.random.default_rng(6)
    q, k, v = r.standard_normal((2, 1, 8)), r.standard_normal((6, 1, 8)), r.standard_normal((6, 1, 8))
    want = oa.tree_attention(q, k, v, 4, [0b1, 0b10], 1.0)
    k[5], v[5] = np.nan, np.inf
    got = oa.tree_attention(q, k, v, 4, [0b1, 0b10], 1.0)
    assert np.array_equal(got[0], want[0]) and np.isnan(got[1]).all()


def test_commit_moves_a_path():
    pos = np.arange(10)
    assert oa.commit(pos, 4, [0, 2, 5]).tolist() == [0, 1, 2, 3, 4, 6, 9, 7, 8, 9]
    assert oa.commit(pos, 4, [0, 1, 2]).tolist() == pos.tolist()
