"""The oracle of tree accept and of cache pages against what they have to be, without a GPU."""

import itertools

import numpy as np
import pytest

from oracle import accept as oa, tree as ot


def dist(r, V, spread=1.5):
    z = r.standard_normal(V) * spread
    p = np.exp(z - z.max())
    return p / p.sum()


@pytest.mark.parametrize("distinct", [False, True])
@pytest.mark.parametrize("V,k", [(3, 1), (4, 2), (5, 3)])
def test_children_leave_the_target_exact(V, k, distinct):
    """Summed over all draws of the children and all decisions, the emitted token has the target's distribution."""
    r = np.random.default_rng(V * 10 + k)
    p, q = dist(r, V), dist(r, V)
    out = np.zeros(V)
    for kids in itertools.product(range(V), repeat=k):
        if distinct and len(set(kids)) < k:
            continue
        chance, left = 1.0, 1.0
        for x in kids:
            chance *= q[x] / left
            left -= q[x] if distinct else 0.0
        steps, last = ot.residuals(p, q, list(kids), distinct)
        for x, (rj, qj) in zip(kids, steps):
            if rj is None:
                break
            a = min(1.0, rj[x] / qj[x])
            out[x] += chance * a
            chance *= 1 - a
        out += chance * (last if last is not None else p)
    assert np.abs(out - p).max() < 1e-12


def test_chain_is_the_chain_rule():
    r = np.random.default_rng(3)
    for _ in range(200):
        m, V = int(r.integers(0, 5)), 11
        z = (r.standard_normal((m + 1, V)) * 2).astype(np.float32)
        q = np.stack([dist(r, V) for _ in range(m + 1)]).astype(np.float32)
        draft = [int(r.choice(V, p=q[i] / q[i].astype(np.float64).sum())) for i in range(m)]
        u = r.random(m + 1).astype(np.float32)
        n, tokens = oa.sampled_accept(z, q[:m], draft, 0.8, np.concatenate([u[1:], u[:1]]))
        path, got, _ = ot.accept(z, [-1] + list(range(m)), [0] + draft, 0.8, q, u)
        assert got == list(tokens) and len(path) == n and path == list(range(n))


def test_drafts_without_a_distribution_follow_the_target():
    r = np.random.default_rng(4)
    z = (r.standard_normal((4, 5)) * 2).astype(np.float32)
    for _ in range(50):
        u = r.random(4).astype(np.float32)
        path, tokens, _ = ot.accept(z, [-1, 0, 0, 1], [0, 2, 3, 1], 1.0, None, u)
        p = ot.target(z[0], 1.0)
        first = int(np.searchsorted(np.cumsum(p), float(u[0]) * p.sum(), side="right"))
        assert tokens[0] == first and (len(path) > 1) == (first in (2, 3))


def test_truncation_keeps_the_shortest_prefix():
    z = np.array([1.0, 3.0, 3.0, -2.0, 0.5], dtype=np.float32)
    p = ot.target(z, 1.0, top_k=2)
    assert np.nonzero(p)[0].tolist() == [1, 2]
    p = ot.target(z, 1.0, top_k=1)
    assert np.nonzero(p)[0].tolist() == [1]                   # the lower index of two alike
    whole = ot.target(z, 1.0)
    p = ot.target(z, 1.0, top_p=0.9)
    kept = np.nonzero(p)[0]
    order = np.lexsort((np.arange(5), -z))
    share = np.cumsum(whole[order]) / whole.sum()
    assert len(kept) == 1 + int(np.sum(share < np.float32(0.9)))


def test_pages_model_keeps_its_counts():
    r = np.random.default_rng(5)
    page, slots, n = 4, 5, 40
    m = ot.Pages(n, page, slots, 10)
    length = [0] * slots
    for _ in range(300):
        what = r.integers(0, 4)
        if what == 0:
            p, c = (int(x) for x in r.choice(slots, 2, replace=False))
            if m.held[c] == 0 and m.held[p]:
                t = int(r.integers(0, length[p] + 1))
                assert m.fork([p], [c], [t]) == [True]
                length[c] = t
        elif what == 1:
            live, moves = m.compact()
            assert all(p < live for s in range(slots) for p in m.table[s][:m.held[s]]) and all(a >= live > b for a, b in moves)
        else:
            keep = [int(r.integers(0, length[s] + 1)) if r.random() < 0.3 else length[s] for s in range(slots)]
            need = [k + int(r.integers(0, 9)) if r.random() < 0.7 else (0 if k == 0 else k) for k in keep]
            need = [-1 if r.random() < 0.2 else min(x, 40) for x in need]
            keep = [min(k, x) if x >= 0 else k for k, x in zip(keep, need)]
            missing, copies, fresh = m.reserve(keep, need)
            if not missing:
                for s in range(slots):
                    if need[s] >= 0:
                        length[s] = need[s]
                        for e in range(keep[s] // page, m.held[s]):
                            assert m.refs[m.table[s][e]] == 1
        count = [0] * n
        for s in range(slots):
            for p in m.table[s][:m.held[s]]:
                count[p] += 1
        assert count == m.refs
