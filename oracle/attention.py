"""The steps between a layer's q|k|v and o projections, in fp64.

[reading] The pages give no layer internals; these are the usual ones of the
target family: RMS norm of each head, rotary positions, a KV cache (bf16, or
affine codes in the weight format) and softmax attention in which a drafted
row sees every committed token and its own ancestors among the drafts.
"""

import numpy as np

GROUP = 64
KV_FAR = np.float32(65280.0)   # inputs are clamped to it, so scale * code + bias stays inside fp16


def norm_rope(x, weight, eps, norm, positions, inv_freq, interleaved):
    """fp64 [rows, heads, dim] from x [rows, heads, dim] (values of bf16 inputs), one rounding away from the output."""
    y = np.asarray(x, dtype=np.float64).copy()
    if norm:
        y /= np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps)
        if weight is not None:
            y *= np.asarray(weight, dtype=np.float64)
    if inv_freq is None or not len(inv_freq):
        return y
    half = len(inv_freq)
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    j = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    u, v = y[..., i].copy(), y[..., j].copy()
    y[..., i] = u * c - v * s
    y[..., j] = v * c + u * s
    return y


def kv_quantize(x, bits):
    """(codes int [..., dim], scales fp16, biases fp16 [..., dim / 64]) of fp32 values, the format's own roundings."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    bad = np.isnan(g).any(axis=-1)
    g = np.clip(np.where(bad[..., None], np.float32(0), g), -KV_FAR, KV_FAR)
    lo, hi = g.min(axis=-1), g.max(axis=-1)
    top = np.float32(2 ** bits - 1)
    s = ((hi - lo) / top).astype(np.float16)
    b = lo.astype(np.float16)
    s32 = s.astype(np.float32)[..., None]
    step = (g - b.astype(np.float32)[..., None]) / np.where(s32 == 0, np.float32(1), s32)
    codes = np.where(s32 == 0, 0, np.clip(np.rint(step), 0, top)).astype(np.int64)
    s, b = np.where(bad, np.float16(np.nan), s), np.where(bad, np.float16(np.nan), b)
    codes = np.where(bad[..., None], 0, codes)
    return codes.reshape(x.shape), s, b


def kv_dequantize(codes, s, b):
    """fp64 values of codes [..., dim]."""
    return codes * np.repeat(s.astype(np.float64), GROUP, axis=-1) + np.repeat(b.astype(np.float64), GROUP, axis=-1)


def pack(codes, bits):
    """uint32 words [..., dim * bits / 32], least significant field first."""
    per = 32 // bits
    c = np.asarray(codes, dtype=np.uint64).reshape(codes.shape[:-1] + (codes.shape[-1] // per, per))
    return (c << (np.arange(per, dtype=np.uint64) * np.uint64(bits))).sum(axis=-1).astype(np.uint32)


def unpack(words, bits):
    per = 32 // bits
    w = np.asarray(words, dtype=np.uint32)[..., None] >> (np.arange(per, dtype=np.uint32) * np.uint32(bits))
    return (w & np.uint32(2 ** bits - 1)).astype(np.int64).reshape(words.shape[:-1] + (words.shape[-1] * (32 // bits),))


def chain_masks(m):
    return [(1 << (i + 1)) - 1 for i in range(m)]


def visible(m, length, masks):
    """bool [m, length + m]: what each drafted row sees."""
    seen = np.ones((m, length + m), dtype=bool)
    for i in range(m):
        for j in range(m):
            seen[i, length + j] = bool(masks[i] >> j & 1)
    return seen


def tree_attention(q, k, v, length, masks, scale):
    """fp64 [m, q_heads, dim]: q [m, q_heads, dim] over k, v [length + m, kv_heads, dim]; a row that sees nothing is zero.

    Sums run over the visible tokens only, so what a row does not see cannot reach it."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    m, heads, dim = q.shape
    group = heads // k.shape[1]
    seen = visible(m, length, masks)
    out = np.zeros((m, heads, dim))
    for i in range(m):
        at = np.nonzero(seen[i])[0]
        if not len(at):
            continue
        for h in range(heads):
            z = scale * (k[at, h // group] @ q[i, h])
            top = z.max()
            if top == -np.inf:
                continue
            p = np.exp(z - top)
            out[i, h] = (p @ v[at, h // group]) / p.sum()
    return out


def commit(positions, length, path):
    """Where each position of a request's sequence comes from after the accepted path moved up."""
    src = np.asarray(positions).copy()
    for j, i in enumerate(path):
        src[length + j] = positions[length + i]
    return src
