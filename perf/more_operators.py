"""Cases, plain forms and exact values of the operators of a batch that shares a prompt and drafts trees.

* ``share``   attention of drafted rows over a prefix that the requests of a group have in common, and over each request's own
              tokens (sv_tree_attention_shared)
* ``accept``  verification of a draft tree against the target's probabilities, from given uniforms (sv_tree_accept)
* ``round``   the pages of a batch over one round: children forked from a prompt, what they will write reserved (the half-filled
              page is copied), the children freed again (sv_kv_fork, sv_kv_reserve)
* ``compact`` live pages moved to the front of the cache (sv_kv_compact)
* ``copy``    pages handed from one cache to another (sv_kv_copy_pages)

Heads come from the dense targets of this repository: 32 query and 8 key heads (hidden 4096 and 2560), 48 and 8 (hidden
5120), 128 wide; 64 wide heads are generic.  Vocabularies are 151936 and generic ones.
"""

import math

import torch

own = False

GROUP = 64
LEAST = 2.0 ** -24   # of the draft's mass that is left once its tried tokens are taken out

_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        from speculative_decoding_verify_qmm_gb300 import binding
        _LIB = binding.load()
    return _LIB


# ------------------------------------------------------------------- cases

def listed():
    return [
        # four samples of one short prompt, one token each: the smallest call, latency-bound
        dict(name="share_token", op="share", batch=4, groups=1, rows=1, ragged=False, hq=32, hk=8, d=128, bits=16, page=64,
             prefix=1024, own=130, tree="chain"),
        # sixteen chats behind one 16K system prompt, 8 drafted rows each, 8-bit cache
        dict(name="share_chat", op="share", batch=16, groups=1, rows=8, ragged=False, hq=32, hk=8, d=128, bits=8, page=64,
             prefix=16384, own=700, tree="chain"),
        # 64 samples in plain decoding over 4-bit codes in small pages, an odd number of pages in common
        dict(name="share_decode", op="share", batch=64, groups=1, rows=1, ragged=False, hq=32, hk=8, d=128, bits=4, page=16,
             prefix=8016, own=2011, tree="chain"),
        # two long documents, twelve requests with 32-node trees on each, in a 48-head layer: bound by the tensor cores
        dict(name="share_tree", op="share", batch=24, groups=2, rows=32, ragged=True, hq=48, hk=8, d=128, bits=16, page=128,
             prefix=30000, own=1500, tree="tree"),
        # greedy trees of four requests, from raw logits
        dict(name="accept_greedy", op="accept", batch=4, nodes=16, ragged=False, vocab=151936, mode="greedy", stats=False,
             top_k=0, top_p=1.0),
        # one request's 32-node tree, children drawn without replacement, the head's row statistics at hand
        dict(name="accept_one", op="accept", batch=1, nodes=32, ragged=False, vocab=151936, mode="distinct", stats=True,
             top_k=0, top_p=1.0),
        # a large batch of wide trees, children drawn independently, from raw logits
        dict(name="accept_batch", op="accept", batch=24, nodes=64, ragged=True, vocab=151936, mode="independent", stats=False,
             top_k=0, top_p=1.0),
        # a draft of most likely tokens (no distribution) against a truncated target
        dict(name="accept_top", op="accept", batch=8, nodes=24, ragged=False, vocab=151936, mode="target", stats=True,
             top_k=64, top_p=0.95),
        # eight samples of one 5000-token prompt set up for a round of 8 rows, 36 layers of 8-bit codes
        dict(name="pages_fork", op="round", slots=8, prompts=1, rows=8, layers=36, hk=8, d=128, bits=8, page=64, length=5000,
             spare=40),
        # 96 samples of three prompts, in 64 layers of a bf16 cache
        dict(name="pages_batch", op="round", slots=96, prompts=3, rows=32, layers=64, hk=8, d=128, bits=16, page=16,
             length=1511, spare=500),
        # a third of a 4-bit cache's pages are free after requests have left: the live ones move to the front
        dict(name="pages_compact", op="compact", slots=40, pages=3000, live=0.67, layers=36, hk=8, d=128, bits=4, page=16),
        # a prompt's pages handed to another cache (a decoding engine's) in 36 layers
        dict(name="pages_copy", op="copy", pages=300, moved=257, layers=36, hk=8, d=128, bits=8, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["share", "share", "share", "accept", "accept", "accept", "round", "compact", "copy"])
    d, page, hk = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 8])
    bits = rng.choice([4, 8, 16])
    if op == "share":
        batch, rows, hq = _log_int(rng, 2, 128), _log_int(rng, 1, 64), hk * rng.randint(1, 8)
        # rows x heads x tokens stay below the largest listed case's
        most = max(page, min(40000, 24 * 16 * 48 * 30000 // (batch * rows * hq)))
        return dict(op=op, batch=batch, groups=rng.randint(1, min(3, batch)), rows=rows, ragged=rng.random() < 0.5, hq=hq, hk=hk,
                    d=d, bits=bits, page=page, prefix=_log_int(rng, page, most), own=_log_int(rng, 1, min(2500, most)),
                    tree=rng.choice(["chain", "tree"]))
    if op == "accept":
        mode, nodes = rng.choice(["greedy", "distinct", "independent", "target"]), _log_int(rng, 1, 64)
        cut = rng.random() < 0.3
        return dict(op=op, batch=min(24, max(1, _log_int(rng, 1, 1200) // nodes)), nodes=nodes, ragged=rng.random() < 0.5,
                    vocab=rng.choice([32000, 151936, rng.randint(1000, 200000)]), mode=mode, stats=rng.random() < 0.5,
                    top_k=rng.choice([0, 20, 200]) if cut else 0, top_p=rng.choice([0.8, 0.95]) if cut else 1.0)
    c = dict(op=op, layers=_log_int(rng, 1, 64), hk=hk, d=d, bits=bits, page=page)
    pages = max(4, _log_int(rng, 4, 3000) * 16 // page)
    if op == "round":
        slots = _log_int(rng, 2, 96)
        c |= dict(slots=slots, prompts=rng.randint(1, min(4, slots - 1)), rows=_log_int(rng, 1, 64), length=rng.randint(1, 3000),
                  spare=slots * (2 + 64 // page) + rng.randint(0, 50))
        pages = c["prompts"] * -(-c["length"] // page) + c["spare"]
    elif op == "compact":
        c |= dict(slots=_log_int(rng, 1, 64), pages=pages, live=rng.uniform(0.2, 0.95))
    else:
        c |= dict(pages=pages, moved=rng.randint(1, pages))
    c["layers"] = max(1, min(c["layers"], 2500000000 // (pages * _stored(c, page))))          # of the largest listed caches' size
    return c


def _counts(case):
    """Rows (nodes) of each request: all alike, or spread from 1 to the case's number."""
    B, n = case["batch"], case["rows" if case["op"] == "share" else "nodes"]
    return [1 + (n - 1) * ((b * 7 + 3) % B) // max(1, B - 1) if case["ragged"] and B > 1 else n for b in range(B)]


def _offsets(counts):
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + c)
    return offs


def _share_plan(case):
    """(first request of each group, pages that each group shares, committed tokens of each request)."""
    B, G, page = case["batch"], case["groups"], case["page"]
    first = [g * B // G for g in range(G + 1)]
    pages = [max(1, (case["prefix"] - case["prefix"] * g // (3 * G)) // page) for g in range(G)]
    group = [max(g for g in range(G) if first[g] <= b) for b in range(B)]
    lens = [pages[group[b]] * page + case["own"] - case["own"] * ((b * 5) % B) * 4 // (5 * B) for b in range(B)]
    return first, pages, lens


def _stored(case, tokens):
    """Bytes that `tokens` tokens take in one layer's cache."""
    row = 2 * case["hk"] * case["d"]
    return tokens * (row * 2 if case["bits"] == 16 else row * case["bits"] // 8 + row // GROUP * 4)


def work(case):
    op = case["op"]
    if op == "share":
        first, pages, lens = _share_plan(case)
        counts, page = _counts(case), case["page"]
        common = sum(pages) * page
        alone = sum(lens) + sum(counts) - sum(pages[g] * page * (first[g + 1] - first[g]) for g in range(case["groups"]))
        pairs = sum((n + c) * c for n, c in zip(lens, counts))
        return {"bytes": _stored(case, common + alone) + 4 * sum(counts) * case["hq"] * case["d"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    if op == "accept":
        # the row that the last token comes from; with a draft's distribution, that row of it too
        rows = 2 if case["mode"] in ("distinct", "independent") else (0 if case["mode"] == "greedy" and case["stats"] else 1)
        return {"bytes": case["batch"] * (4 * rows * case["vocab"] + 16 * case["nodes"]), "flops": 4 * case["batch"] * case["vocab"]}
    if op == "round":
        part = case["length"] % case["page"]
        return {"bytes": 2 * (case["slots"] - case["prompts"]) * case["layers"] * _stored(case, part) + 24 * case["slots"], "flops": 0}
    if op == "compact":
        n, live = case["pages"], _live(case)
        moved = n - live - sum(1 for i in range(live, n) if not _is_live(case, i))
        return {"bytes": 2 * moved * case["layers"] * _stored(case, case["page"]) + 8 * n, "flops": 0}
    return {"bytes": 2 * case["moved"] * case["layers"] * _stored(case, case["page"]), "flops": 0}


def _is_live(case, i):
    return (i * 2654435761 >> 7) % 1000 < 1000 * case["live"]


def _live(case):
    return sum(_is_live(case, i) for i in range(case["pages"]))


# ------------------------------------------------------------------ inputs

def _quantize(x, bits):
    """(packed words int32 [..., D * bits / 32], scales, biases fp16 [..., D / 64]) of fp32 values [..., D]."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s, b = ((hi - lo) / (2 ** bits - 1)).half(), lo.half()
    code = torch.round((g - b.float()) / s.float()).clamp(0, 2 ** bits - 1)
    code = torch.where(s == 0, 0.0, code).to(torch.int64).flatten(-2).unflatten(-1, (-1, 32 // bits))
    words = (code << (bits * torch.arange(32 // bits, device=x.device))).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), s.squeeze(-1), b.squeeze(-1)


def _dequantize(words, s, b, bits):
    """fp32 values [..., D] of packed words."""
    shifts = bits * torch.arange(32 // bits, device=words.device, dtype=torch.int32)
    code = ((words.unsqueeze(-1) >> shifts) & (2 ** bits - 1)).flatten(-2).unflatten(-1, (-1, GROUP))
    return (code.float() * s.unsqueeze(-1).float() + b.unsqueeze(-1).float()).flatten(-2)


def _filled(gen, n_pages, hk, page, d, bits):
    """A cache of seeded values: a dict of its tensors."""
    parts = {}
    for name in ("k", "v"):
        x = torch.randn((n_pages, hk, page, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        if bits == 16:
            parts[name] = x
        else:
            parts[name], parts[name + "_scales"], parts[name + "_biases"] = _quantize(x.float(), bits)
    return parts


def _layers(gen, case, n_pages):
    """Caches of several layers: a dict of tensors [layers, ...], any bytes will do for copies."""
    L, hk, page, d, bits = case["layers"], case["hk"], case["page"], case["d"], case["bits"]
    parts = {}
    for name in ("k", "v"):
        if bits == 16:
            parts[name] = torch.randn((L, n_pages, hk, page, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        else:
            parts[name] = torch.randint(-2 ** 31, 2 ** 31 - 1, (L, n_pages, hk, page, d * bits // 32), generator=gen,
                                        device="cuda", dtype=torch.int32)
            for t in ("_scales", "_biases"):
                parts[name + t] = torch.randn((L, n_pages, hk, page, d // GROUP), generator=gen, device="cuda").half()
    return parts


def _handles(parts):
    lib = _lib()
    return lib.kv_layers([lib.kv_cache(**{n: t[i] for n, t in parts.items()}) for i in range(parts["k"].shape[0])])


def _ancestors(gen, counts):
    """Random trees: row i > 0 hangs below an earlier row; bit j of a row's word is set for itself and its ancestors."""
    rnd = torch.rand(sum(counts), generator=gen, device="cuda").tolist()
    words, at = [], 0
    for n in counts:
        mine = []
        for i in range(n):
            parent = int(rnd[at + i] * i) if i else -1
            mine.append((mine[parent] if parent >= 0 else 0) | (1 << i))
        words += mine
        at += n
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64, device="cuda")


def _prepare_share(case, gen):
    s = {"case": case}
    page, hk, d, B = case["page"], case["hk"], case["d"], case["batch"]
    first, shared, lens = _share_plan(case)
    counts = _counts(case)
    offs = _offsets(counts)
    n_own = [-(-(n + c) // page) for n, c in zip(lens, counts)]
    table = torch.full((B, max(n_own)), -1, dtype=torch.int32, device="cuda")
    group = [max(g for g in range(case["groups"]) if first[g] <= b) for b in range(B)]
    total = sum(shared) + sum(n - shared[g] for n, g in zip(n_own, group))
    perm = torch.randperm(total + 3, generator=gen, device="cuda").to(torch.int32)
    at = 0
    for g, n in enumerate(shared):
        table[first[g]:first[g + 1], :n] = perm[at:at + n]
        at += n
    for b in range(B):
        n = n_own[b] - shared[group[b]]
        table[b, shared[group[b]]:n_own[b]] = perm[at:at + n]
        at += n
    s["table"], s["parts"] = table, _filled(gen, total + 3, hk, page, d, case["bits"])
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q"] = (torch.randn((offs[-1], case["hq"] * d), generator=gen, device="cuda") * 2).to(torch.bfloat16)
    s["tree"] = _ancestors(gen, counts) if case["tree"] == "tree" else None
    if own:
        lib = _lib()
        s["cache"] = lib.kv_cache(**s["parts"])
        s["groups"], s["offsets"] = lib.prefix_groups(first, shared), lib.row_offsets(offs)
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = lib.workspace(lib.tree_attention_shared_workspace_bytes(s["cache"], s["groups"], s["offsets"], case["hq"]))
    return s


def _prepare_accept(case, gen):
    s = {"case": case, "T": 0.0 if case["mode"] == "greedy" else 0.75}
    V, mode, counts = case["vocab"], case["mode"], _counts(case)
    offs = _offsets(counts)
    rows = offs[-1]
    rnd = torch.rand((rows, 2), generator=gen, device="cuda").tolist()
    parent, nth = [], []
    for b, n in enumerate(counts):            # trees up to 10 deep with up to 4 children a node, new ones often under late nodes
        depth, kids = [0], [0]
        parent.append(-1)
        nth.append(0)
        for i in range(1, n):
            r = rnd[offs[b] + i]
            free = [v for v in range(i) if kids[v] < 4 and depth[v] < 10]
            v = free[int(len(free) * (r[0] ** 0.5 if r[1] < 0.6 else r[0]))] if free else i - 1
            parent.append(v)
            nth.append(kids[v])
            kids[v] += 1
            kids.append(0)
            depth.append(depth[v] + 1)
    s["parent"] = torch.tensor(parent, dtype=torch.int32, device="cuda")
    s["offs"] = torch.tensor(offs, dtype=torch.int64, device="cuda")
    base = torch.repeat_interleave(s["offs"][:-1], s["offs"][1:] - s["offs"][:-1])
    above = base + s["parent"].clamp(min=0)   # the row of each node's parent
    s["logits"] = torch.randn((rows, V), generator=gen, device="cuda") * 2.5
    draft = s["logits"] + torch.randn((rows, V), generator=gen, device="cuda") * 0.7
    nth = torch.tensor(nth, device="cuda")
    if mode in ("greedy", "target"):          # a node's children are the draft's most likely tokens, in order
        top = draft.topk(4 if mode == "target" else 2, dim=1).indices
        s["tokens"] = top[above, nth.clamp(max=top.shape[1] - 1)].to(torch.int32)
        s["q"] = None
    else:
        s["q"] = torch.softmax(draft / s["T"], 1)
        del draft
        if mode == "distinct":                # the largest of perturbed log-probabilities: draws without replacement
            noise = -torch.log(-torch.log(torch.rand((rows, V), generator=gen, device="cuda").clamp(1e-30, 1 - 2 ** -24)))
            s["tokens"] = (torch.log(s["q"]) + noise).topk(4, dim=1).indices[above, nth].to(torch.int32)
        else:
            cum = s["q"].double().cumsum(1)[above]
            at = torch.rand((rows, 1), generator=gen, device="cuda", dtype=torch.float64) * cum[:, -1:]
            s["tokens"] = torch.searchsorted(cum, at, right=True).clamp(max=V - 1).squeeze(1).to(torch.int32)
            del cum
    s["u"] = torch.rand(rows, generator=gen, device="cuda")
    s["depth"] = 11
    s["stats"] = None
    if case["stats"]:                         # what the head leaves beside the logits
        top, arg = s["logits"].max(1)
        z = ((s["logits"] - top[:, None]).double() / max(s["T"], 1e-9)) if s["T"] else torch.zeros((rows, 1), device="cuda")
        s["stats"] = (top, torch.exp(z).sum(1).float(), arg.to(torch.int32))
    if own:
        lib = _lib()
        s["offsets"] = lib.row_offsets(offs)
        s["out"] = (torch.zeros(len(counts), dtype=torch.int32, device="cuda"), torch.full((rows,), -1, dtype=torch.int32, device="cuda"),
                    torch.full((len(counts), max(counts)), -1, dtype=torch.int32, device="cuda"))
        s["workspace"] = lib.workspace(lib.tree_accept_workspace_bytes(rows))
    s["most"] = max(counts)
    return s


def _prepare_round(case, gen, seed):
    s = {"case": case}
    page, slots, prompts, n = case["page"], case["slots"], case["prompts"], case["length"]
    held = -(-n // page)
    n_pages = prompts * held + case["spare"]
    s["parts"] = _layers(gen, case, n_pages)
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    s["table"] = torch.full((slots, -(-(n + case["rows"]) // page)), -1, dtype=torch.int32, device="cuda")
    s["table"][:prompts, :held] = perm[:prompts * held].view(prompts, held)
    s["refs"] = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    s["refs"][perm[:prompts * held].long()] = 1
    s["held"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
    s["held"][:prompts] = held
    kids = torch.arange(prompts, slots, device="cuda")
    s["child"], s["parent"] = kids.to(torch.int32), (kids % prompts).to(torch.int32)
    s["tokens"] = torch.full_like(s["child"], n)
    s["keep"] = torch.full((slots,), n, dtype=torch.int32, device="cuda")
    s["need"] = s["keep"] + case["rows"]
    s["none"] = torch.zeros_like(s["keep"])
    s["leave"] = torch.where(torch.arange(slots, device="cuda") < prompts, s["keep"], 0)      # the children go, the prompts stay
    if own:
        lib = _lib()
        s["layers"] = _handles(s["parts"])
        s["pages"] = lib.kv_pages(s["refs"], s["table"], s["held"], page)
        s["workspace"] = lib.workspace(lib.kv_reserve_workspace_bytes(s["pages"]))
        s["counts"], s["copies"] = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty((slots, 3), dtype=torch.int32, device="cuda")
    return s


def _prepare_compact(case, gen, seed):
    s = {"case": case}
    n, slots = case["pages"], case["slots"]
    s["parts"] = _layers(gen, case, n)
    live = torch.tensor([i for i in range(n) if _is_live(case, i)], dtype=torch.int64, device="cuda")
    live = live[torch.randperm(len(live), generator=gen, device="cuda")]
    per = -(-max(1, len(live)) // slots)
    table = torch.full((slots * (per + 1),), -1, dtype=torch.int32, device="cuda").view(slots, per + 1)
    padded = torch.full((slots * per,), -1, dtype=torch.int32, device="cuda")
    padded[:len(live)] = live.to(torch.int32)
    table[:, 1:] = padded.view(slots, per)
    if len(live):
        table[:, 0] = live[0].to(torch.int32)                                                  # one page that everybody shares
    s["table0"] = table
    s["held"] = (table >= 0).sum(1).to(torch.int32)
    s["refs0"] = torch.zeros(n, dtype=torch.int32, device="cuda").scatter_add_(
        0, table.clamp(min=0).flatten().long(), (table >= 0).flatten().to(torch.int32))
    s["table"], s["refs"] = torch.empty_like(table), torch.empty_like(s["refs0"])
    if own:
        lib = _lib()
        s["layers"] = _handles(s["parts"])
        s["pages"] = lib.kv_pages(s["refs"], s["table"], s["held"], case["page"])
        s["counts"], s["moves"] = torch.empty(2, dtype=torch.int32, device="cuda"), torch.empty((n, 2), dtype=torch.int32, device="cuda")
    return s


def _prepare_copy(case, gen, seed):
    s = {"case": case}
    n, m = case["pages"], case["moved"]
    s["parts"], s["to"] = _layers(gen, case, n), _layers(gen, case, n)
    s["src"] = torch.randint(0, n, (m,), generator=gen, device="cuda").to(torch.int32)         # the same page twice is fine
    s["dst"] = torch.randperm(n, generator=gen, device="cuda")[:m].to(torch.int32)
    if own:
        s["layers"], s["layers_to"] = _handles(s["parts"]), _handles(s["to"])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op == "share":
        return _prepare_share(case, gen)
    if op == "accept":
        return _prepare_accept(case, gen)
    return {"round": _prepare_round, "compact": _prepare_compact, "copy": _prepare_copy}[op](case, gen, seed)


# -------------------------------------------------------------- plain forms

def _values(s, name, pages):
    """fp32 values [..., hk, tokens, d] of rows of pages [..., n]."""
    p = s["parts"]
    x = p[name][pages].float() if s["case"]["bits"] == 16 else \
        _dequantize(p[name][pages], p[name + "_scales"][pages], p[name + "_biases"][pages], s["case"]["bits"])
    return x.transpose(-4, -3).flatten(-3, -2)


def _plain_share(s):
    c = s["case"]
    hq, hk, d, page = c["hq"], c["hk"], c["d"], c["page"]
    first, shared, _ = _share_plan(c)
    counts = _counts(c)
    offs = _offsets(counts)
    outs = []
    for g in range(c["groups"]):
        b0, b1, n = first[g], first[g + 1], shared[g]
        r0, r1, most = offs[b0], offs[b1], max(counts[b0:b1])
        offsets = torch.tensor(offs[b0:b1 + 1], device="cuda")
        row = offsets[:-1, None] + torch.arange(most, device="cuda")                                 # [requests, most]
        real = row < offsets[1:, None]
        row = torch.where(real, row, r0)
        q = s["q"].float().unflatten(1, (hk, hq // hk, d))
        # the common pages, once for all rows of the group
        kc, vc = (_values(s, t, s["table"][b0, :n].long()) for t in ("k", "v"))                        # [hk, tokens, d]
        qc = q[r0:r1].transpose(0, 1).flatten(1, 2)                                                    # [hk, rows * heads, d]
        sc = torch.matmul(qc, kc.transpose(-1, -2)) * (d ** -0.5)
        # each request's own tokens and drafts
        ko, vo = (_values(s, t, s["table"][b0:b1, n:].long().clamp(min=0)) for t in ("k", "v"))        # [requests, hk, tokens, d]
        qo = q[row].permute(0, 2, 1, 3, 4).flatten(2, 3)                                               # [requests, hk, most * heads, d]
        so = torch.matmul(qo, ko.transpose(-1, -2)) * (d ** -0.5)
        back = n * page + torch.arange(ko.shape[2], device="cuda") - s["kv_len"][b0:b1, None]          # place among the drafts
        if s["tree"] is None:
            seen = back[:, None, :] <= torch.arange(most, device="cuda")[:, None]
        else:
            bit = (s["tree"][row][:, :, None] >> back.clamp(0, 63)[:, None, :]) & 1
            seen = (back < 0)[:, None, :] | ((bit == 1) & (back < 64)[:, None, :])
        so = torch.where(seen.repeat_interleave(hq // hk, 1)[:, None], so, -math.inf)
        # both parts of a row under one maximum: the own part of the padded rows goes back to the rows' order
        back_rows = lambda x: x.unflatten(2, (most, hq // hk)).permute(0, 2, 1, 3, 4)[real].transpose(0, 1).flatten(1, 2)  # noqa: E731
        top = torch.maximum(sc.amax(-1, keepdim=True), back_rows(so.amax(-1, keepdim=True)))
        pad = torch.zeros((b1 - b0, most, hk, hq // hk, 1), device="cuda")
        pad[real] = top.unflatten(1, (r1 - r0, hq // hk)).transpose(0, 1)
        pc = torch.exp(sc - top)
        po = torch.exp(so - pad.permute(0, 2, 1, 3, 4).flatten(2, 3))
        o = torch.matmul(pc, vc) + back_rows(torch.matmul(po, vo))
        o = o / (pc.sum(-1, keepdim=True) + back_rows(po.sum(-1, keepdim=True)))
        outs.append(o.unflatten(1, (r1 - r0, hq // hk)).transpose(0, 1).flatten(1).to(torch.bfloat16))
    return torch.cat(outs)


def _kept(z, top, T, top_k, top_p):
    """Which tokens of logit rows [n, V] a truncated target keeps: largest first, ties to the lower index."""
    V = z.shape[1]
    order = torch.sort(z, dim=1, descending=True, stable=True).indices
    w = torch.exp((z.gather(1, order) - top[:, None]).double() / T)
    rank = torch.arange(V, device=z.device)
    w = torch.where(rank < (top_k or V), w, 0.0)
    before = w.cumsum(1) - w
    kept = (rank < (top_k or V)) & (before < top_p * w.sum(1, keepdim=True) if top_p < 1 else torch.ones_like(w, dtype=torch.bool))
    return torch.zeros_like(kept).scatter_(1, order, kept)


def _plain_accept(s):
    c = s["case"]
    T, V, B, most = s["T"], c["vocab"], c["batch"], s["most"]
    offs = s["offs"]
    first, n = offs[:-1], offs[1:] - offs[:-1]
    at = torch.arange(B, device="cuda")
    node = torch.arange(most, device="cuda")
    real = node < n[:, None]
    rows = torch.where(real, first[:, None] + node, 0)                                    # [B, most]
    parent = torch.where(real & (node > 0), s["parent"].long()[rows], -2)
    same = (parent[:, :, None] == parent[:, None, :]) & (node[None, :] < node[:, None])    # an earlier row with the same parent
    nth = same.sum(2)
    tokens, u = s["tokens"].long()[rows], s["u"].double()[rows]
    out_len = torch.zeros(B, dtype=torch.int32, device="cuda")
    out_tokens = torch.full((s["u"].shape[0],), -1, dtype=torch.int32, device="cuda")
    path = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    v, live = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.ones(B, dtype=torch.bool, device="cuda")
    length = torch.ones(B, dtype=torch.int64, device="cuda")
    for _ in range(min(most, s["depth"])):
        r = first + v
        z = s["logits"][r]
        child = parent == v[:, None]
        if not T:
            want = z.argmax(1) if s["stats"] is None else s["stats"][2][r].long()
            drawn, hit = want, child & (tokens == want[:, None])
            found, took = hit.any(1), hit.to(torch.int8).argmax(1)
        else:
            top = z.amax(1) if s["stats"] is None else s["stats"][0][r]
            E = torch.exp((z.double() - top.double()[:, None]) / T)
            if c["top_k"] or c["top_p"] < 1:
                E = torch.where(_kept(z, top, T, c["top_k"], c["top_p"]), E, 0.0)
                M = E.sum(1)
            else:
                M = E.sum(1) if s["stats"] is None else s["stats"][1][r].double()
            W, took, found = E, torch.zeros_like(v), torch.zeros_like(live)
            if s["q"] is not None:
                q, left = s["q"][r].double(), torch.ones(B, dtype=torch.float64, device="cuda")
                for j in range(4):
                    mine = child & (nth == j)
                    k = mine.to(torch.int8).argmax(1)
                    x = tokens[at, k]
                    fits = u[at, k] * q[at, x] * M < W[at, x] * left
                    ask = mine.any(1) & live & ~found
                    found, took = found | (ask & fits), torch.where(ask & fits, k, took)
                    no = (ask & ~fits)[:, None]
                    W = torch.where(no, (W - (M / left)[:, None] * q).clamp(min=0), W)
                    M = torch.where(no[:, 0], W.sum(1), M)
                    if c["mode"] == "distinct":
                        left = torch.where(no[:, 0], (left - q[at, x]).clamp(min=LEAST), left)
                        q = torch.where(no, q.scatter(1, x[:, None], 0.0), q)
                W = torch.where((M > 0)[:, None], W, E)
            cum = W.cumsum(1)
            theta = (u[:, 0] if s["q"] is not None else u[at, v]) * cum[:, -1]
            drawn = torch.searchsorted(cum, theta[:, None], right=True).squeeze(1).clamp(max=V - 1)
            if s["q"] is None:
                hit = child & (tokens == drawn[:, None])
                found, took = hit.any(1), hit.to(torch.int8).argmax(1)
        emitted = torch.where(found, tokens[at, took], drawn)
        place = torch.where(live, first + length - 1, first)
        out_tokens[place] = torch.where(live, emitted.to(torch.int32), out_tokens[place])
        out_len = torch.where(live, length, out_len.long()).to(torch.int32)
        live = live & found
        v = torch.where(live, took, v)
        spot = torch.where(live, length, 0)
        path[at, spot] = torch.where(live, took.to(torch.int32), path[at, spot])
        length = length + live
    return out_len, out_tokens, path


def _plain_reserve(s, keep, need):
    """Every slot holds ceil(need / page) pages, alone from token `keep` on; the lowest free pages, in slot and entry order."""
    c, table, refs, held = s["case"], s["table"], s["refs"], s["held"]
    page, (slots, width) = c["page"], table.shape
    entry, has, wants = torch.arange(width, device="cuda"), held.long()[:, None], (need.long()[:, None] + page - 1) // page
    keep = keep.long()[:, None]
    pages = torch.where(entry < has, table.long(), 0)
    shared = (refs[pages] > 1) & (entry < has)
    part = (keep % page > 0) & (entry == keep // page) & (entry < has)
    # the half-filled page of several slots: where all that name it ask for it, the first of them keeps it
    asks = torch.where(part & shared, pages, -1).amax(1)
    alike = (asks[:, None] == asks[None, :]) & (asks >= 0)[:, None]
    keeps = (alike.sum(1) == refs[asks.clamp(min=0)]) & ~(alike & (torch.arange(slots, device="cuda") < torch.arange(slots, device="cuda")[:, None])).any(1)
    copied = part & shared & ~keeps[:, None]
    fresh = (entry < wants) & ((entry >= has) | copied | (shared & ~part & (entry >= keep // page)))
    free = refs == 0
    lowest = torch.argsort(torch.where(free, 0, 1), stable=True)
    rank = fresh.flatten().cumsum(0) - 1
    new = lowest[rank.clamp(min=0)].view(slots, width)
    gone = ((entry < has) & (fresh | (entry >= wants))).flatten()
    refs.scatter_add_(0, pages.flatten(), -gone.to(torch.int32))
    refs.scatter_add_(0, torch.where(fresh, new, 0).flatten(), fresh.flatten().to(torch.int32))
    table.copy_(torch.where(fresh, new.to(torch.int32), table))
    held.copy_(wants.squeeze(1).to(torch.int32))
    return pages[copied], new[copied]                                       # one page at most of a slot


def _plain_copy(s, to, src, dst, places):
    for name, t in s["parts"].items():
        to[name][:, dst, :, :places] = t[:, src, :, :places]


def _plain_round(s):
    c = s["case"]
    page, refs, table, held = c["page"], s["refs"], s["table"], s["held"]
    n = -(-c["length"] // page)
    parents, kids = s["parent"].long(), s["child"].long()
    table[kids, :n] = table[parents, :n]
    refs.scatter_add_(0, table[kids, :n].long().flatten(), torch.ones(len(kids) * n, dtype=torch.int32, device="cuda"))
    held[kids] = -(-s["tokens"] // page)
    src, dst = _plain_reserve(s, s["keep"], s["need"])
    _plain_copy(s, s["parts"], src, dst, c["length"] % page)
    _plain_reserve(s, s["leave"], s["leave"])


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    refs.copy_(s["refs0"])
    table.copy_(s["table0"])
    n = refs.shape[0]
    live = refs > 0
    count = live.sum()
    at = torch.arange(n, device="cuda")
    moving, holes = live & (at >= count), ~live & (at < count)
    src = torch.argsort(torch.where(moving, 0, 1), stable=True)
    dst = torch.argsort(torch.where(holes, 0, 1), stable=True)
    real = at < moving.sum()
    to = at.clone()
    to[src] = torch.where(real, dst, src)
    m = int(moving.sum())                                                                       # pages that move
    _plain_copy(s, s["parts"], src[:m], dst[:m], s["case"]["page"])
    refs.copy_(torch.zeros_like(refs).scatter_add_(0, to, refs))
    entry = torch.arange(table.shape[1], device="cuda")
    table.copy_(torch.where(entry < s["held"][:, None], to[table.long().clamp(min=0)].to(torch.int32), table))


def run(s):
    c = s["case"]
    op = c["op"]
    if op == "share":
        if not own:
            return _plain_share(s)
        return _lib().tree_attention_shared(s["cache"], s["groups"], s["offsets"], s["kv_len"], s["table"], s["q"], c["hq"],
                                            tree_mask=s["tree"], out=s["out"], workspace=s["workspace"])
    if op == "accept":
        if not own:
            return _plain_accept(s)
        return _lib().tree_accept(s["offsets"], s["logits"], s["parent"], s["tokens"], s["T"], q=s["q"], u=s["u"],
                                  distinct=c["mode"] == "distinct", top_k=c["top_k"], top_p=c["top_p"], stats=s["stats"],
                                  out=s["out"], workspace=s["workspace"])
    if op == "round":
        if not own:
            _plain_round(s)
        else:
            lib = _lib()
            lib.kv_fork(s["pages"], s["parent"], s["child"], s["tokens"])
            lib.kv_reserve(s["pages"], s["layers"], s["keep"], s["need"], counts=s["counts"], copies=s["copies"], workspace=s["workspace"])
            lib.kv_reserve(s["pages"], s["layers"], s["leave"], s["leave"], counts=s["counts"], copies=s["copies"], workspace=s["workspace"])
        return s["refs"], s["table"], s["held"], s["parts"]
    if op == "compact":
        if not own:
            _plain_compact(s)
        else:
            s["refs"].copy_(s["refs0"])
            s["table"].copy_(s["table0"])
            _lib().kv_compact(s["pages"], s["layers"], counts=s["counts"], moves=s["moves"])
        return s["refs"], s["table"], s["parts"]
    if not own:
        _plain_copy(s, s["to"], s["src"].long(), s["dst"].long(), c["page"])
    else:
        _lib().kv_copy_pages(s["layers"], s["src"], s["dst"], to=s["layers_to"])
    return s["to"]


# ------------------------------------------------------------- exact values

def _exact_values(words, s, b, bits):
    """fp64 values of int32 code words [..., W], by arithmetic on the words taken as unsigned numbers."""
    u = words.to(torch.int64) % (1 << 32)
    fields = torch.stack([(u // (1 << (bits * j))) % (1 << bits) for j in range(32 // bits)], -1).flatten(-2)
    return fields.double() * s.double().repeat_interleave(GROUP, -1) + b.double().repeat_interleave(GROUP, -1)


def _exact_share(s):
    c, p = s["case"], s["parts"]
    counts, (_, _, lens), d = _counts(c), _share_plan(c), c["d"]
    offs, outs = _offsets(counts), []
    for b in range(c["batch"]):
        n, m = lens[b], counts[b]
        pages = s["table"][b, :-(-(n + m) // c["page"])].long()
        take = lambda t: t.index_select(0, pages).transpose(1, 2).flatten(0, 1)[:n + m]  # noqa: E731
        k, v = (take(p[t]).double() if c["bits"] == 16 else
                _exact_values(take(p[t]), take(p[t + "_scales"]), take(p[t + "_biases"]), c["bits"]) for t in ("k", "v"))
        q = s["q"][offs[b]:offs[b + 1]].double().reshape(m, c["hk"], -1, d)
        hide = torch.zeros((m, n + m), dtype=torch.bool)
        for i in range(m):
            bits = int(s["tree"][offs[b] + i]) if s["tree"] is not None else (1 << (i + 1)) - 1
            hide[i, n:] = torch.tensor([not bits >> j & 1 for j in range(m)])
        z = torch.einsum("mhgd,thd->hgmt", q, k) / math.sqrt(d)
        z = z.masked_fill(hide.cuda()[None, None], -math.inf)
        outs.append(torch.einsum("hgmt,thd->mhgd", torch.softmax(z, -1), v).reshape(m, -1))
    return torch.cat(outs)


def _exact_accept(s):
    """Request after request and node after node, as the rule is written: residuals are normalised at each step."""
    c, T, V = s["case"], s["T"], s["case"]["vocab"]
    parent, tokens, u = s["parent"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    offs = s["offs"].tolist()
    out_len, out_tokens, paths = [], [-1] * offs[-1], []
    for b in range(c["batch"]):
        r0, n = offs[b], offs[b + 1] - offs[b]
        kids = [[i for i in range(1, n) if parent[r0 + i] == v] for v in range(n)]
        v, path = 0, [0]
        while True:
            z = s["logits"][r0 + v].double()
            took = None
            if not T:
                drawn = int(s["logits"][r0 + v].argmax())
                took = next((i for i in kids[v] if tokens[r0 + i] == drawn), None)
            else:
                p = torch.softmax(z / T, 0)
                if c["top_k"] or c["top_p"] < 1:
                    order = torch.sort(s["logits"][r0 + v], descending=True, stable=True).indices[:c["top_k"] or V]
                    mass = p[order].cumsum(0)
                    count = int((mass - p[order] < c["top_p"] * mass[-1]).sum()) if c["top_p"] < 1 else len(order)
                    kept = torch.zeros_like(p)
                    kept[order[:count]] = p[order[:count]]
                    p = kept / kept.sum()
                rest = p
                if s["q"] is not None:
                    q = s["q"][r0 + v].double()
                    gone = 0.0
                    for i in kids[v]:
                        x = tokens[r0 + i]
                        now = q / max(1.0 - gone, LEAST)
                        if u[r0 + i] * float(now[x]) < float(rest[x]):
                            took = i
                            break
                        rest = (rest - now).clamp(min=0)
                        if float(rest.sum()) > 0:
                            rest = rest / rest.sum()
                        if c["mode"] == "distinct":
                            gone += float(q[x])
                            q[x] = 0
                    rest = rest if float(rest.sum()) > 0 else p
                cum = rest.cumsum(0)
                drawn = int((cum <= (u[r0] if s["q"] is not None else u[r0 + v]) * float(cum[-1])).sum().clamp(max=V - 1))
                if s["q"] is None:
                    took = next((i for i in kids[v] if tokens[r0 + i] == drawn), None)
            out_tokens[r0 + len(path) - 1] = drawn if took is None else tokens[r0 + took]
            if took is None:
                break
            path.append(took)
            v = took
        out_len.append(len(path))
        paths.append(path + [-1] * (s["most"] - len(path)))
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda") for x in (out_len, out_tokens, paths))


def _exact_round(s):
    """Page after page on the host: fork, reserve, free."""
    c = s["case"]
    page, n, rows = c["page"], c["length"], c["rows"]
    refs, table, held = s["refs"].tolist(), s["table"].tolist(), s["held"].tolist()
    full, part = n // page, n % page
    moves = []
    for kid, up in zip(s["child"].tolist(), s["parent"].tolist()):
        held[kid] = -(-n // page)
        for e in range(held[kid]):
            table[kid][e] = table[up][e]
            refs[table[kid][e]] += 1
    free = [i for i, r in enumerate(refs) if r == 0]
    for slot in range(c["slots"]):
        if part and slot >= c["prompts"]:                       # the prompt itself is the first that names its last page
            moves.append((table[slot][full], free[0]))
            refs[table[slot][full]] -= 1
            refs[free[0]] = 1
            table[slot][full] = free.pop(0)
        for e in range(held[slot], -(-(n + rows) // page)):
            refs[free[0]] = 1
            table[slot][e] = free.pop(0)
        held[slot] = -(-(n + rows) // page)
    for slot in range(c["slots"]):
        stay = -(-n // page) if slot < c["prompts"] else 0
        for e in range(stay, held[slot]):
            refs[table[slot][e]] -= 1
        held[slot] = stay
    parts = {k: t.clone() for k, t in s["parts"].items()}
    for a, b in moves:
        for k, t in s["parts"].items():
            parts[k][:, b, :, :part] = t[:, a, :, :part]
    whole = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (refs, table, held)]
    return (*whole, {k: t.double() if t.is_floating_point() else t for k, t in parts.items()})


def _exact_compact(s):
    refs, table, held = s["refs0"].tolist(), s["table0"].tolist(), s["held"].tolist()
    live = sum(r > 0 for r in refs)
    holes = [i for i in range(live) if refs[i] == 0]
    to = {p: holes[i] for i, p in enumerate(p for p in range(live, len(refs)) if refs[p])}
    parts = {k: t.clone() for k, t in s["parts"].items()}
    for a, b in to.items():
        refs[b], refs[a] = refs[a], 0
        for k, t in s["parts"].items():
            parts[k][:, b] = t[:, a]
    table = [[to.get(p, p) if e < held[i] else p for e, p in enumerate(row)] for i, row in enumerate(table)]
    whole = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (refs, table)]
    return (*whole, {k: t.double() if t.is_floating_point() else t for k, t in parts.items()})


def _exact_copy(s):
    parts = {k: t.clone() for k, t in s["to"].items()}
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for k, t in s["parts"].items():
            parts[k][:, b] = t[:, a]
    return {k: t.double() if t.is_floating_point() else t for k, t in parts.items()}


def exact(case, seed):
    return {"share": _exact_share, "accept": _exact_accept, "round": _exact_round, "compact": _exact_compact,
            "copy": _exact_copy}[case["op"]](prepare(case, seed))
