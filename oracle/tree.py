"""The accept step of a draft tree, and the pages of a cache, written out step by step.

[reading] The pages state the accept rule for a chain (mlx-dspark releases page, v0.0.2 "Highlights": accept with probability
min(1, p / q), resample the residual).  A tree applies it at each node to the children in turn: the first on p, each further one on what
the rejected ones left, so that the output stays an exact sample of the target; drafts without a distribution are followed where the
target's own draw falls on them.  Nothing here is shared with the GPU code: residuals are normalised at each step, in fp64.
"""

import numpy as np

LEAST = 2.0 ** -24          # of the draft's mass that is left once its tried tokens are taken out
UNIT = 2.0 ** -40           # what a weight is counted in, of the largest


def target(z, temperature, top_k=0, top_p=1.0):
    """fp64 probabilities of a row, truncated: largest logit first, ties to the lower index."""
    z = np.asarray(z, dtype=np.float32).astype(np.float64)
    w = np.exp((z - z.max()) / np.float64(np.float32(temperature)))
    order = np.lexsort((np.arange(len(z)), -z))
    keep = order[:top_k] if 0 < top_k < len(z) else order
    if top_p < 1:
        cum = np.cumsum(w[keep])
        keep = keep[:int(np.sum(cum - w[keep] < np.float64(np.float32(top_p)) * cum[-1]))]
    out = np.zeros_like(w)
    out[keep] = w[keep]
    return out


def residuals(p, q, tokens, distinct):
    """[(r_j, q_j)] for each child's token in turn, if all before it are rejected, and the r that is left after the last.

    r is normalised, or None where nothing is left; q_j is None for a token tried before without replacement."""
    r, out, gone = p / p.sum(), [], []
    for x in tokens:
        if distinct and x in gone:
            out.append((r, None))
            continue
        qj = np.asarray(q, dtype=np.float64).copy()
        qj[gone] = 0.0
        left = 1.0
        for g in gone:
            left = max(left - float(q[g]), LEAST)
        qj /= left
        out.append((r, qj))
        if r is not None:
            r = np.maximum(0.0, r - qj)
            r = r / r.sum() if r.sum() > 0 else None
        if distinct:
            gone = gone + [x]
    return out, r


def accept(logits, parent, token, temperature, q=None, u=None, distinct=False, top_k=0, top_p=1.0, max_path=64, sumexp=None):
    """(path, tokens, margin) of one request.  margin: how near the nearest decision was to going the other way, as a share of the weight
    decided on, with the share that counting in units may move it taken off; below 0 it may have gone either way."""
    n, V = len(parent), len(logits[0])
    v, path, tokens, margin = 0, [0], [], np.inf
    while True:
        kids = [i for i in range(1, n) if parent[i] == v] if len(path) < max_path else []
        took = None
        if not temperature:
            drawn = int(np.argmax(logits[v]))
            took = next((i for i in kids if token[i] == drawn), None)
        else:
            w = target(logits[v], temperature, top_k, top_p)
            total = w.sum() if sumexp is None else float(sumexp[v])
            slack = 8 * (len(kids) + 1) * V * UNIT / max(w.sum(), 1e-300) + 1e-11
            p = w / total
            r = p
            if q is not None:
                steps, last = residuals(w, q[v], [token[i] for i in kids], distinct)
                if sumexp is not None and kids:                 # p is not normalised exactly: its own sum stands for 1
                    steps, last = _given(p, q[v], [token[i] for i in kids], distinct)
                r = p / p.sum() if not kids else last
                for i, (rj, qj) in zip(kids, steps):
                    if qj is None:
                        continue
                    x = token[i]
                    a, b = float(np.float32(u[i])) * float(qj[x]), 0.0 if rj is None else float(rj[x])
                    margin = min(margin, abs(a - b) - slack)
                    if a < b:
                        took = i
                        break
            if took is None:
                if r is None:
                    r = p
                cum = np.cumsum(r)
                theta = float(np.float32(u[0] if q is not None else u[v])) * cum[-1]
                drawn = int(np.searchsorted(cum, theta, side="right"))
                drawn = min(drawn, int(np.nonzero(r > 0)[0][-1]))
                near = np.abs(cum - theta)
                margin = min(margin, near.min() / cum[-1] - slack)
                if q is None:
                    took = next((i for i in kids if token[i] == drawn), None)
        tokens.append(int(token[took]) if took is not None else drawn)
        if took is None:
            return path, tokens, margin
        path.append(took)
        v = took


def _given(p, q, tokens, distinct):
    """residuals() of a p that is taken as it is for the first test."""
    steps, last = residuals(p, q, tokens, distinct)
    out, r, gone, left = [], p, [], 1.0
    for x, (_, qj) in zip(tokens, steps):
        out.append((r, qj))
        if qj is None:
            continue
        if r is not None:
            r = np.maximum(0.0, r - qj)
            r = r / r.sum() if r.sum() > 0 else None
    return out, r


class Pages:
    """Who has which page, and what each page's places hold in every layer (any hashable value)."""

    def __init__(self, n_pages, page, slots, width):
        self.page, self.refs, self.held = page, [0] * n_pages, [0] * slots
        self.table = [[0] * width for _ in range(slots)]
        self.places = [[None] * page for _ in range(n_pages)]

    def fork(self, parents, children, tokens):
        """The forks that are made, as truth values."""
        done = []
        for f, (p, c, t) in enumerate(zip(parents, children, tokens)):
            ok = 0 <= p < len(self.held) and 0 <= c < len(self.held) and t >= 0 and p not in children and c not in children[:f]
            n = -(-t // self.page)
            ok = ok and self.held[c] == 0 and n <= self.held[p]
            done.append(ok)
            if ok:
                for e in range(n):
                    self.table[c][e] = self.table[p][e]
                    self.refs[self.table[p][e]] += 1
                self.held[c] = n
        return done

    def reserve(self, keep, need):
        """(pages missing, copies, fresh pages)."""
        page, slots = self.page, range(len(self.held))
        active = [s for s in slots if need[s] >= 0]
        half = {s: self.table[s][keep[s] // page] for s in active if keep[s] % page}
        half = {s: p for s, p in half.items() if self.refs[p] > 1}
        copied = {s for s, p in half.items() if not (self.refs[p] == sum(v == p for v in half.values()) and s == min(t for t, v in half.items() if v == p))}
        fresh = []
        for s in active:
            for e in range(keep[s] // page, -(-need[s] // page)):
                part = keep[s] % page and e == keep[s] // page
                if e >= self.held[s] or (s in copied if part else self.refs[self.table[s][e]] > 1):
                    fresh.append((s, e))
        free = [i for i, r in enumerate(self.refs) if r == 0]
        if len(free) < len(fresh):
            return len(fresh) - len(free), [], 0
        copies, gone = [], []
        for (s, e), new in zip(fresh, free):
            if e < self.held[s]:
                gone.append(self.table[s][e])
                if keep[s] % page and e == keep[s] // page:
                    copies.append((self.table[s][e], new, keep[s] % page))
            self.table[s][e] = new
            self.refs[new] = 1
        for s in active:
            n = -(-need[s] // page)
            gone += [self.table[s][e] for e in range(n, self.held[s])]
            self.held[s] = n
        for p in gone:
            self.refs[p] -= 1
        for a, b, n in copies:
            self.places[b][:n] = self.places[a][:n]
        return 0, copies, len(fresh)

    def compact(self):
        """(pages in use, moves)."""
        live = sum(r > 0 for r in self.refs)
        holes = [i for i in range(live) if self.refs[i] == 0]
        moves = list(zip([i for i in range(live, len(self.refs)) if self.refs[i]], holes))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.places[b] = list(self.places[a])
        for s, n in enumerate(self.held):
            self.table[s][:n] = [to.get(p, p) for p in self.table[s][:n]]
        return live, moves
