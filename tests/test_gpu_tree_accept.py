"""Accept of draft trees against the fp64 oracle.

Decisions are equal unless one is nearer to its border than the arithmetic may move it: a weight exp((z - max) / T) is off by at most
about one unit of 2^-40 of the largest, a product A q by another, A itself (a sum over the vocabulary) by V of them, so a cumulative sum
of the j-th residual is off by less than 8 (j + 1) V units.  The oracle returns how far its nearest decision is from that.  A decision
inside it has two right answers: a draw among 20,000 tokens meets a border each 5e-5, of which 16 V 2^-40 = 3e-7 are inside, so about one
decision of 170, and such a request is only checked for being a path of its tree.
"""

import numpy as np
import pytest
import torch

from oracle import tree as ot
from speculative_decoding_verify_qmm_gb300.binding import SVError

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def softmax(z):
    w = np.exp(z.astype(np.float64) - z.max(-1, keepdims=True))
    return w / w.sum(-1, keepdims=True)


class Case:
    """Random trees: logits, a draft near them, children drawn from it (or its likeliest tokens where q is None)."""

    def __init__(self, seed, counts, V, T, mode, spread=2.0, noise=0.6, kids=4):
        r = np.random.default_rng(seed)
        self.counts, self.V, self.T, self.mode = counts, V, T, mode
        rows = sum(counts)
        self.offs = [0] + np.cumsum(counts).tolist()
        self.z = (r.standard_normal((rows, V)) * spread).astype(np.float32)
        draft = self.z + r.standard_normal((rows, V)).astype(np.float32) * np.float32(noise)
        self.q = softmax(draft / (T or 1.0)).astype(np.float32) if mode in ("independent", "distinct") else None
        self.parent, self.token = np.full(rows, -1, np.int32), np.full(rows, -7, np.int32)   # the anchor's are not read
        order = np.argsort(-draft, axis=1)
        for b, n in enumerate(counts):
            o, children = self.offs[b], [[] for _ in range(n)]
            for i in range(1, n):
                v = int(r.choice([v for v in range(i) if len(children[v]) < min(kids, V)]))
                self.parent[o + i] = v
                if self.q is None:
                    x = order[o + v][len(children[v])]
                else:
                    p = self.q[o + v].astype(np.float64)
                    if mode == "distinct":
                        p[children[v]] = 0
                    x = r.choice(V, p=p / p.sum())
                children[v].append(int(x))
                self.token[o + i] = x
        self.u = r.random(rows).astype(np.float32)

    def stats(self):
        top = self.z.max(1)
        T = np.float64(np.float32(self.T)) if self.T else 1.0
        with np.errstate(over="ignore"):
            return top, np.exp((self.z - top[:, None]).astype(np.float64) / T).sum(1).astype(np.float32), self.z.argmax(1).astype(np.int32)

    def call(self, lib, stats=False, **kw):
        st = tuple(dev(x) for x in self.stats()) if stats else None
        return lib.tree_accept(self.offs, dev(self.z), dev(self.parent), dev(self.token), self.T, q=None if self.q is None else dev(self.q),
                               u=dev(self.u) if self.T else None, distinct=self.mode == "distinct", stats=st, **kw)

    def check(self, out, stats=False, top_k=0, top_p=1.0, max_path=64, sure=True):
        length, tokens, path = (t.cpu().numpy() for t in out)
        sums = self.stats()[1] if stats and top_k == 0 and top_p == 1 and self.T else None
        for b, n in enumerate(self.counts):
            s = slice(self.offs[b], self.offs[b] + n)
            want, emitted, margin = ot.accept(self.z[s], self.parent[s].tolist(), self.token[s].tolist(), self.T,
                                              None if self.q is None else self.q[s], self.u[s], self.mode == "distinct", top_k, top_p, max_path,
                                              None if sums is None else sums[s])
            if margin < 0:
                assert 1 <= length[b] <= n and path[b, 0] == 0 and not (sure and self.V <= 4097)
                assert all(self.parent[s][path[b, i]] == path[b, i - 1] for i in range(1, length[b]))
                continue
            assert length[b] == len(want), (b, length[b], want, margin)
            assert path[b, :len(want)].tolist() == want and (path[b, len(want):] == -1).all()
            assert tokens[s][:len(want)].tolist() == emitted and (tokens[s][len(want):] == -1).all(), (b, tokens[s], emitted, margin)


MODES = ["greedy", "independent", "distinct", "target"]


@pytest.mark.parametrize("stats", [False, True])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("counts,V", [([1], 2), ([2, 1, 3], 3), ([7, 64, 1, 20], 17), ([33, 32, 31], 1000), ([12] * 5, 4097), ([40, 3], 50001)])
def test_trees(lib, counts, V, mode, stats):
    for seed in range(4 if V < 20000 else 2):
        c = Case(seed * 100 + V + len(mode), counts, V, 0.0 if mode == "greedy" else 0.7, mode, kids=3 if V == 3 else 4)
        c.check(c.call(lib, stats), stats)
    assert lib.device_error() == 0


@pytest.mark.parametrize("mode", ["independent", "distinct", "target"])
@pytest.mark.parametrize("top_k,top_p", [(1, 1.0), (5, 1.0), (0, 0.8), (40, 0.9), (700, 1.0), (0, 0.999)])
def test_truncated_targets(lib, mode, top_k, top_p):
    for seed, V in ((1, 33), (2, 1000), (3, 20011)):
        c = Case(seed + top_k, [9, 24, 1], V, 0.9, mode)
        for stats in (False, True):
            c.check(c.call(lib, stats, top_k=top_k, top_p=top_p), stats, top_k=min(top_k, V) if top_k < V else 0, top_p=top_p)
    assert lib.device_error() == 0


def test_flat_rows_truncated_by_count_and_mass(lib):
    """More candidates than are sorted: ties by index, and the places found bit by bit."""
    V = 20000
    for spread, top_k, top_p in ((0.0, 6000, 1.0), (1e-3, 9000, 0.7), (1e-3, 0, 0.6), (0.0, 0, 0.5), (0.01, 5000, 1.0)):
        for mode in ("target", "independent"):
            c = Case(11, [4, 1], V, 1.0, mode, spread=spread, noise=0.1)
            c.check(c.call(lib, top_k=top_k, top_p=top_p), top_k=top_k, top_p=top_p)


def test_ties_take_the_lowest_index(lib):
    V = 3000
    c = Case(5, [6, 6], V, 0.0, "greedy")
    c.z[:] = np.float32(-1.0)
    c.z[:, 700], c.z[:, 2900] = 2.0, 2.0
    c.z[:, 5] = -0.0
    c.parent[:] = [-1, 0, 0, 1, 1, 4] * 2
    c.token[:] = [0, 2900, 700, 700, 700, 700] * 2             # two children with one token: the first is followed
    c.parent[6:] = [-1, 0, 0, 1, 2, 2]
    c.check(c.call(lib))
    length, _, path = c.call(lib)
    assert path[0, :2].tolist() == [0, 2] and path[1, :3].tolist() == [0, 2, 4]


def test_a_chain_is_accepted_as_by_spec_accept(lib):
    for seed in range(6):
        c = Case(seed, [9, 1, 5], 2000, 0.8, "independent")
        for b, n in enumerate(c.counts):                         # the same drafts as a chain
            c.parent[c.offs[b]:c.offs[b] + n] = np.arange(-1, n - 1)
        r = np.random.default_rng(seed)
        for b, n in enumerate(c.counts):
            for i in range(1, n):
                c.token[c.offs[b] + i] = r.choice(c.V, p=softmax(np.log(c.q[c.offs[b] + i - 1])))
        length, tokens, path = c.call(lib)
        keep = np.concatenate([np.arange(c.offs[b], c.offs[b + 1] - 1) for b in range(3)]).astype(np.int64)
        u = np.concatenate([np.roll(c.u[c.offs[b]:c.offs[b + 1]], -1) for b in range(3)])
        want_len, want = lib.spec_accept_batched(c.offs, dev(c.z), dev(c.token[keep + 1]), c.T, q=dev(c.q[keep]), u=dev(u))
        assert torch.equal(length, want_len) and torch.equal(tokens, want)


def test_zero_draft_probability_and_no_residual(lib):
    """p == q leaves no residual (never reached by a test that can fail: u just below 1); q(x) == 0 is accepted where p(x) > 0."""
    V, T = 64, 1.0
    c = Case(1, [3], V, T, "independent")
    c.parent[:] = [-1, 0, 0]
    c.q[0] = 0
    c.q[0, 10] = 1.0                                             # both drafts came with probability 0
    c.token[:] = [0, 7, 9]
    length, tokens, path = c.call(lib)
    assert path[0].tolist()[:2] == [0, 1] and tokens[0] == 7
    # a target with one token, a draft with another: rejected, and the residual is the target
    c.z[:] = -np.inf
    c.z[:, 33] = 0.0
    c.token[:] = [0, 10, 10]
    length, tokens, path = c.call(lib)
    assert length.item() == 1 and tokens[0] == 33
    # p is q exactly and the draft is rejected by a u of 1 - 2^-24 times q against p smaller by its rounding: the draw is from p
    c = Case(2, [2], 4, 1.0, "independent")
    c.z[:] = 0.0
    c.q[:] = 0.5
    c.token[:] = [0, 2]
    c.u[:] = [0.6, 1 - 2.0 ** -24]
    length, tokens, path = c.call(lib)                           # W = max(0, 1/4 - 1/2) = 0 everywhere
    assert length.item() == 1 and tokens[0].item() == 2
    assert lib.device_error() == 0


def test_children_with_one_token_without_replacement(lib):
    c = Case(3, [5], 50, 0.8, "distinct")
    c.parent[:] = [-1, 0, 0, 0, 0]
    x = int(np.argsort(c.z[0])[5])
    c.token[:] = [0, x, x, x, int(np.argmax(c.z[0]))]
    c.q[0] = softmax(-c.z[0] / 0.8)
    c.u[1:] = 0.99
    c.check(c.call(lib))


@pytest.mark.parametrize("mode", MODES)
def test_infinite_logits_and_extreme_uniforms(lib, mode):
    c = Case(8, [6, 6, 6], 900, 0.0 if mode == "greedy" else 1.3, mode)
    c.z[:, ::2] = -np.inf
    c.z[:, 1] += 40.0
    for u in (0.0, 2.0 ** -24, 0.5, 1 - 2.0 ** -24):
        c.u[:] = u
        c.check(c.call(lib), sure=u == 0.5)               # the other u lie on borders
        _, tokens, _ = c.call(lib, stats=True)
        assert all(t % 2 == 1 for t in tokens.tolist() if t != -1)   # no token without weight, at any u


def test_rows_without_any_weight_stay_in_range(lib):
    """NaN, all -inf, +inf: the tokens mean nothing, but they are tokens, and nothing hangs."""
    for fill in (np.nan, -np.inf, np.inf):
        for mode in MODES:
            c = Case(9, [4, 2], 700, 0.0 if mode == "greedy" else 1.0, mode)
            c.z[0] = fill
            for kw in ({}, dict(top_k=7), dict(top_p=0.5)):
                length, tokens, path = c.call(lib, **kw)
                assert 1 <= length[0] <= 4 and 0 <= tokens[0] < 700
                ref = Case(9, [4, 2], 700, c.T, mode).call(lib, **kw)
                assert torch.equal(tokens[4:], ref[1][4:])       # the other request does not notice


@pytest.mark.parametrize("max_path", [1, 2, 3, 64])
def test_max_path_ends_the_walk(lib, max_path):
    for mode in MODES:
        c = Case(12, [10, 10], 300, 0.0 if mode == "greedy" else 0.5, mode, noise=0.05, kids=1)
        if mode == "greedy":
            for b in range(2):
                for i in range(1, 10):
                    c.token[c.offs[b] + i] = c.z[c.offs[b] + i - 1].argmax()
        out = c.call(lib, max_path=max_path)
        assert out[2].shape == (2, max_path)
        c.check(out, max_path=max_path)


@pytest.mark.parametrize("V", [400001, 1 << 19])
@pytest.mark.parametrize("mode", ["independent", "distinct", "target"])
def test_large_vocabularies(lib, V, mode):
    """Slices that shared memory does not hold."""
    c = Case(13, [5, 3], V, 0.6, mode, spread=3.0)
    c.check(c.call(lib), sure=False)
    c.check(c.call(lib, top_k=100, top_p=0.9), top_k=100, top_p=0.9, sure=False)


def test_largest_vocabulary_and_batch(lib):
    z = torch.zeros((2, 1 << 22), device="cuda")
    z[0, 4000000], z[1, 3] = 30.0, 30.0
    tok = torch.tensor([0, 4000000], dtype=torch.int32, device="cuda")
    par = torch.tensor([-1, 0], dtype=torch.int32, device="cuda")
    length, tokens, path = lib.tree_accept([0, 2], z, par, tok, 0.5, u=torch.full((2,), 0.5, device="cuda"))
    assert length.item() == 2 and tokens.tolist() == [4000000, 3]
    counts = [1 + b % 7 for b in range(256)]
    for mode in MODES:
        c = Case(14, counts, 130, 0.0 if mode == "greedy" else 1.0, mode)
        c.check(c.call(lib))


def test_strides_and_untouched_outputs(lib):
    c = Case(15, [6, 3], 333, 0.8, "independent")
    z, q = torch.full((11, 400), 9.0, device="cuda"), torch.full((11, 350), 9.0, device="cuda")
    z[:9, :333], q[:9, :333] = dev(c.z), dev(c.q)
    out = (torch.full((4,), -1, dtype=torch.int32, device="cuda"), torch.full((12,), -1, dtype=torch.int32, device="cuda"),
           torch.full((3, 9), -1, dtype=torch.int32, device="cuda"))
    got = lib.tree_accept(c.offs, z[:, :333], dev(c.parent), dev(c.token), c.T, q=q[:, :333], u=dev(c.u), out=out)
    c.check((got[0], got[1][:9], got[2]))
    assert (out[0][2:] == -1).all() and (out[1][9:] == -1).all() and (out[2][2:] == -1).all()
    odd = torch.zeros(9 * 333 + 1, device="cuda")                # rows that begin at no particular alignment
    odd[1:] = dev(c.z).flatten()
    got = lib.tree_accept(c.offs, odd[1:].view(9, 333), dev(c.parent), dev(c.token), c.T, q=dev(c.q), u=dev(c.u))
    c.check(got)


@pytest.mark.parametrize("bad", [dict(parent=(2, 2)), dict(parent=(2, 5)), dict(parent=(1, -1)), dict(token=(3, -1)), dict(token=(3, 300))])
def test_bad_trees_are_flagged_and_alone(lib, bad):
    c = Case(16, [5, 5], 300, 0.8, "independent")
    for name, (i, value) in bad.items():
        getattr(c, name)[i] = value
    lib.device_error()
    length, tokens, path = c.call(lib)
    assert lib.device_error() == 4
    assert length[0] == 0 and (tokens[:5] == -1).all() and (path[0] == -1).all()
    good = Case(16, [5, 5], 300, 0.8, "independent")
    ref = good.call(lib)
    assert torch.equal(length[1], ref[0][1]) and torch.equal(tokens[5:], ref[1][5:]) and torch.equal(path[1], ref[2][1])


def test_reproducible_in_a_graph_and_on_two_streams(lib):
    cases = [Case(20 + i, [20, 7], 30011, 0.8, ("distinct", "independent")[i]) for i in range(2)]
    args = [dict(z=dev(c.z), p=dev(c.parent), t=dev(c.token), q=dev(c.q), u=dev(c.u)) for c in cases]

    def run(i, stream=None, out=None, **kw):
        a = args[i]
        return lib.tree_accept(cases[i].offs, a["z"], a["p"], a["t"], 0.8, q=a["q"], u=a["u"], distinct=i == 0, stream=stream, out=out, **kw)
    want = [run(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[run(i, streams[i]) for _ in range(8)] for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for o in got[i] for a, b in zip(o, want[i]))
    out = tuple(torch.full_like(t, -1) for t in want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(0, out=out)
        run(0, out=out, top_k=50)
    for _ in range(2):
        args[0]["u"].copy_(dev(np.random.default_rng(_).random(27).astype(np.float32)))
        for t in out:
            t.fill_(-1)
        g.replay()
        ref = tuple(torch.full_like(t, -1) for t in out)
        run(0, out=ref)
        run(0, out=ref, top_k=50)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_emitted_tokens_have_the_target_distribution(lib):
    """256 requests a call with one tree shape: the first token against softmax(z / T), chi-square."""
    r = np.random.default_rng(30)
    V, T, B, rounds = 16, 0.9, 256, 24
    z = (r.standard_normal(V) * 1.5).astype(np.float32)
    q = softmax((z + r.standard_normal(V).astype(np.float32)) / T).astype(np.float32)
    p = softmax(z / np.float32(T))
    for mode in ("independent", "distinct"):
        seen = np.zeros(V)
        for _ in range(rounds):
            parent = np.tile(np.array([-1, 0, 0, 0], np.int32), B)
            token = np.zeros((B, 4), np.int32)
            qd = q.astype(np.float64) / q.astype(np.float64).sum()
            if mode == "independent":
                token[:, 1:] = r.choice(V, (B, 3), p=qd)
            else:
                token[:, 1:] = np.argsort(-(np.log(qd) + r.gumbel(size=(B, V))), axis=1)[:, :3]
            _, tokens, _ = lib.tree_accept(list(range(0, 4 * B + 1, 4)), dev(np.tile(z, (4 * B, 1))), dev(parent), dev(token.reshape(-1)), T,
                                           q=dev(np.tile(q, (4 * B, 1))), u=dev(r.random(4 * B).astype(np.float32)), distinct=mode == "distinct")
            seen += np.bincount(tokens.view(B, 4)[:, 0].cpu().numpy(), minlength=V)
        n = B * rounds
        chi = ((seen - n * p) ** 2 / (n * p)).sum()
        assert chi < 50.0                                        # 15 degrees of freedom: 1 - 1e-5 lies at 49.3


@pytest.mark.parametrize("mode", ["independent", "distinct", "target"])
@pytest.mark.parametrize("T", [1e-44, 1e-20, 1e5, 2.0 ** 120])
def test_extreme_temperatures_and_logits(lib, mode, T):
    c = Case(40, [7, 12], 600, 1.0, mode)
    c.T = T
    c.z[3, ::3], c.z[4, 5], c.z[4, 6] = -3e38, 3e38, -3e38
    for stats in (False, True):
        for kw in ({}, dict(top_k=9), dict(top_p=0.5)):
            c.check(c.call(lib, stats, **kw), stats, **kw)
    assert lib.device_error() == 0


@pytest.mark.parametrize("mode", MODES)
def test_a_chain_of_64_nodes_that_fits(lib, mode):
    """The deepest path: every draft is the target's certain token."""
    c = Case(41, [64, 64], 200, 0.0 if mode == "greedy" else 1.0, mode, kids=1)
    for b in range(2):
        for i in range(1, 64):
            v = c.offs[b] + i - 1
            c.parent[v + 1], c.token[v + 1] = i - 1, (7 * i) % 200
            c.z[v, (7 * i) % 200] = 90.0
            if c.q is not None:
                c.q[v] = 0.0
                c.q[v, (7 * i) % 200] = 1.0
    length, tokens, path = c.call(lib)
    assert length.tolist() == [64, 64] and path[1].tolist() == list(range(64)) and tokens[64:127].tolist() == [(7 * i) % 200 for i in range(1, 64)]
    c.check((length, tokens, path))


def test_refusals_of_tensors(lib):
    c = Case(17, [3], 100, 0.8, "independent")
    with pytest.raises(SVError):
        c.q = c.q.astype(np.float64)
        c.call(lib)
    c = Case(17, [3], 100, 0.8, "independent")
    with pytest.raises(SVError):
        lib.tree_accept([0, 3], dev(c.z).T.contiguous().T, dev(c.parent), dev(c.token), 0.8, q=dev(c.q), u=dev(c.u))
    with pytest.raises(SVError):
        lib.tree_accept([0, 3], dev(c.z), dev(c.parent)[:2], dev(c.token), 0.8, q=dev(c.q), u=dev(c.u))
    with pytest.raises(SVError):
        lib.tree_accept([0, 3], dev(c.z), dev(c.parent), dev(c.token), 0.8, q=dev(c.q))
    with pytest.raises(SVError):
        lib.tree_accept([0, 0, 3], dev(c.z), dev(c.parent), dev(c.token), 0.8, q=dev(c.q), u=dev(c.u))
