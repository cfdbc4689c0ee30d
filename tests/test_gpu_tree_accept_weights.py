"""The weights that tree accept counts in, to two units of 2^-40 of the largest.

A draw shows a weight through its residual.  Three tokens: the weight in question, the largest, and a rejected draft without weight.  The
head's sum is given as 1, so after that rejection the residuals are E - q_0 and 1 - q_1, where q_0 is the fp32 number near E - 2^-24 and q_1
is 1 - 2^-24: in units, r (some 2^15 to 2^17) and R = 2^16, both subtractions exact.  The first token is drawn iff u < r / (r + R), and near one half
neighbouring uniforms are 2^-6 units of r apart.  A weight is off by 1.25 units at most: its exponent's two floats by 2^-44 ln 2 of the weight, the first
term of 2^(N/128) 2^r to 2^-24 and exactly represented, the rest (below 2^-7.4) rounded some five times, each by 2^-25 of its size,
2^-32.4 in all of which is what the unit of the rest, 2^-41, leaves 0.5, and the last rounding 0.5.  So a uniform below what r - 2 gives draws
the token, and one that r + 2 does not reach does not.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = 2.0 ** -40


def bracket(r, R):
    """fp32 uniforms that decide for any residual of at least r - 2, and against any up to r + 2."""
    lo, hi = (r - 2) / (r - 2 + R), (r + 2) / (r + 2 + R)
    a, b = lo.astype(np.float32), hi.astype(np.float32)
    a = np.where(a.astype(np.float64) >= lo, np.nextafter(a, np.float32(0)), a)
    b = np.where(b.astype(np.float64) < hi, np.nextafter(b, np.float32(1)), b)
    return a, b


@pytest.mark.parametrize("T", [1.0, 0.7, 1.3])
@pytest.mark.parametrize("top", [0.0, 5.3, -40.7])
def test_weights_to_two_units(lib, T, top):
    r = np.random.default_rng(int(10 * T + top + 100))
    n, T32, top32 = 128, float(np.float32(T)), np.float32(top)
    for _ in range(8):
        z = (top32 + np.log(r.uniform(0.07, 0.999, n)) * T).astype(np.float32)
        E = np.exp((z.astype(np.float64) - float(top32)) / T32)
        q0 = (E - 2.0 ** -24).astype(np.float32)
        R = 2.0 ** 16
        left = (E - q0.astype(np.float64)) / UNIT
        assert (left > 2.0 ** 14).all() and (left < 2.0 ** 18).all()
        below, above = bracket(left, R)
        logits, q, u = np.zeros((2 * n, 2, 3), np.float32), np.zeros((2 * n, 2, 3), np.float32), np.full((2 * n, 2), 0.5, np.float32)
        logits[:, :] = [0.0, top32, -np.inf]
        logits[:, 0, 0] = np.repeat(z, 2)
        q[:, 0] = [0.0, 1 - 2.0 ** -24, 0.25]
        q[:, 0, 0] = np.repeat(q0, 2)
        u[0::2, 0], u[1::2, 0] = below, above
        parent, token = np.tile(np.array([-1, 0], np.int32), 2 * n), np.tile(np.array([0, 2], np.int32), 2 * n)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a.reshape(4 * n, -1) if a.ndim == 3 else a.reshape(-1))).cuda()   # noqa: E731
        stats = (torch.full((4 * n,), float(top32), device="cuda"), torch.ones(4 * n, device="cuda"), torch.ones(4 * n, dtype=torch.int32, device="cuda"))
        length, tokens, _ = lib.tree_accept(list(range(0, 4 * n + 1, 2)), dev(logits), dev(parent), dev(token), T, q=dev(q), u=dev(u), stats=stats)
        assert (length == 1).all()
        got = tokens.view(n, 2, 2)[:, :, 0].cpu().numpy()
        assert (got[:, 0] == 0).all() and (got[:, 1] == 1).all(), (np.argwhere(got != [0, 1]), z[(got != [0, 1]).any(1)])
    assert lib.device_error() == 0
