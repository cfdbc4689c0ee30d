"""Cases, plain forms and exact values of the attention-side operators of a verify round.

Four operators stand between a layer's q|k|v projection and its o projection:

* ``rope``    RMS norm of each query and key head with the position rotation (sv_qk_norm_rope)
* ``cache``   the new rows' keys and values written into a paged cache - bf16, or affine 8- / 4-bit codes with
              one fp16 scale and bias per 64 values - and read back (sv_kv_append, sv_kv_read); ``read`` is
              the reading alone, over a long range
* ``attend``  attention of the drafted rows (a chain, or a tree given as ancestor bits) over the cache
              (sv_tree_attention)
* ``commit``  the accepted path's rows moved to the front of the drafted region, all layers at once (sv_kv_commit)

Heads come from the dense targets of this repository: 32 query and 8 key heads (hidden 4096 and 2560), 48 and 8 (hidden
5120), 128 wide; 64 wide heads are generic.
"""

import math

import torch

own = False

GROUP = 64
FAR = 65280.0       # largest bf16 whose group still dequantizes inside fp16's range: inputs are clamped to it
EPS = 1e-6

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
        # one request's 8 drafted rows after the q|k|v projection of a hidden-4096 layer: a launch-bound call
        dict(name="rope_draft", op="rope", rows=8, hq=32, hk=8, d=128, rot=128, interleaved=False, norm=True,
             far=40960),
        # a prompt of odd length in a 48-head layer, far positions, interleaved pairs on half of each head
        dict(name="rope_prompt", op="rope", rows=4093, hq=48, hk=8, d=128, rot=64, interleaved=True, norm=True,
             far=1000000),
        # a continuous batch's round: 4 requests x 8 rows written as 8-bit codes
        dict(name="cache_draft", op="cache", batch=4, rows=8, ragged=False, hk=8, d=128, bits=8, page=64, length=5000),
        # three prompts of different lengths written as 4-bit codes into small pages
        dict(name="cache_prompt", op="cache", batch=3, rows=5501, ragged=True, hk=8, d=128, bits=4, page=16, length=37),
        # a long 8-bit sequence read back (handed to another process, or to a layer that wants bf16)
        dict(name="read_long", op="read", batch=1, rows=32771, ragged=False, hk=8, d=128, bits=8, page=128, length=0),
        # one token of one short request: the plain decode step, latency-bound
        dict(name="attend_token", op="attend", batch=1, rows=1, ragged=False, hq=32, hk=8, d=128, bits=8, page=64,
             length=2047, tree="chain"),
        # the headline round: 8 rows over a 16K context
        dict(name="attend_chain", op="attend", batch=1, rows=8, ragged=False, hq=32, hk=8, d=128, bits=8, page=64,
             length=16384, tree="chain"),
        # a 32-node tree over a long bf16 cache: the widest round
        dict(name="attend_tree", op="attend", batch=1, rows=32, ragged=False, hq=32, hk=8, d=128, bits=16, page=256,
             length=65536, tree="tree"),
        # the continuous batch of 4 x 8 rows in a 48-head layer, contexts of different lengths
        dict(name="attend_batch", op="attend", batch=4, rows=8, ragged=False, hq=48, hk=8, d=128, bits=8, page=64,
             length=30001, tree="tree"),
        # many requests with 1 to 5 rows each over 4-bit codes in small pages
        dict(name="attend_many", op="attend", batch=48, rows=5, ragged=True, hq=32, hk=8, d=128, bits=4, page=16,
             length=12007, tree="tree"),
        # the accepted path of one request's 32-node tree, in all 36 layers
        dict(name="commit_one", op="commit", batch=1, rows=32, path=5, layers=36, hk=8, d=128, page=64),
        # the accepted paths of 24 requests' trees, in 64 layers
        dict(name="commit_batch", op="commit", batch=24, rows=64, path=9, layers=64, hk=8, d=128, page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "read", "attend", "attend", "attend", "commit"])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128, 256])
    if op == "rope":
        hk = rng.choice([1, 2, 8])
        c = dict(op=op, rows=_log_int(rng, 1, 4093), hq=hk * rng.randint(1, 6), hk=hk, d=d,
                 rot=rng.choice([r for r in (32, 64, 96, 128) if r <= d]), interleaved=rng.random() < 0.5,
                 norm=rng.random() < 0.8, far=_log_int(rng, 100, 1000000))
    elif op in ("cache", "read"):
        batch = _log_int(rng, 1, 16)
        c = dict(op=op, batch=batch, rows=max(1, _log_int(rng, 1, 20000) // batch), ragged=rng.random() < 0.5,
                 hk=rng.choice([1, 2, 8]), d=d, bits=rng.choice([4, 8, 16]), page=page, length=rng.randint(0, 3000))
    elif op == "attend":
        batch, rows, hk = _log_int(rng, 1, 48), _log_int(rng, 1, 64), rng.choice([1, 2, 8])
        # rows x heads x tokens stay below the largest listed case's
        hq = hk * rng.randint(1, 6)
        most = min(65536, 32 * 32 * 65536 // (batch * rows * hq), 48 * 8 * 12007 // (batch * hk))
        c = dict(op=op, batch=batch, rows=rows, ragged=rng.random() < 0.5, hq=hq, hk=hk, d=d,
                 bits=rng.choice([4, 8, 16]), page=page, length=_log_int(rng, 1, max(1, most)),
                 tree=rng.choice(["chain", "tree", "tree"]))
    else:
        rows = rng.randint(2, 64)
        c = dict(op=op, batch=_log_int(rng, 1, 24), rows=rows, path=rng.randint(1, min(9, (rows + 1) // 2)),
                 layers=_log_int(rng, 1, 64), hk=rng.choice([1, 2, 8]), d=d, page=page)
    return c


def _counts(case):
    """Rows of each request: all alike, or spread from 1 to the case's number."""
    B, n = case["batch"], case["rows"]
    return [1 + (n - 1) * ((b * 7 + 3) % B) // max(1, B - 1) if case["ragged"] and B > 1 else n for b in range(B)]


def _lengths(case):
    """Committed tokens of each request: the case's length for the first, others spread below it."""
    B, n = case["batch"], case["length"]
    return [n - n * ((b * 5) % B) * 4 // (5 * B) for b in range(B)]


def _offsets(counts):
    offs = [0]
    for c in counts:
        offs.append(offs[-1] + c)
    return offs


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["rows"] * (case["hq"] + case["hk"]) * case["d"]
        return {"bytes": 4 * n, "flops": 7 * n}
    row = 2 * case["hk"] * case["d"]                                  # K and V values of one token
    if op == "commit":
        moved = case["batch"] * (case["path"] - case["path"] // 2) * case["layers"]
        return {"bytes": moved * row * 2 * 2, "flops": 0}
    stored = lambda n: n * (row * 2 if case["bits"] == 16 else row * case["bits"] // 8 + row // GROUP * 4)  # noqa: E731
    rows = sum(_counts(case))
    if op == "cache":  # bf16 rows in, the cache written and read, bf16 rows out
        return {"bytes": 2 * rows * row * 2 + 2 * stored(rows), "flops": 8 * rows * row}
    if op == "read":
        return {"bytes": stored(rows) + rows * row * 2, "flops": 2 * rows * row}
    tokens = [n + c for n, c in zip(_lengths(case), _counts(case))]
    pairs = sum(t * c for t, c in zip(tokens, _counts(case)))
    return {"bytes": sum(stored(t) for t in tokens) + 4 * rows * case["hq"] * case["d"],
            "flops": 4 * pairs * case["hq"] * case["d"]}


# ------------------------------------------------------------------ inputs

def _quantize(x, bits):
    """(packed words int32 [..., D * bits / 32], scales, biases fp16 [..., D / 64]) of fp32 values [..., D].

    The group's scale and bias in fp32, each rounded to fp16; the code is rint((x - bias) / scale)
    with both steps rounded to fp32, clamped to the code's range."""
    g = x.clamp(-FAR, FAR).unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = ((hi - lo) / torch.full_like(hi, float(2 ** bits - 1))).half()
    b = lo.half()
    code = torch.round((g - b.float()) / s.float()).clamp(0, 2 ** bits - 1)
    code = torch.where(s == 0, 0.0, code).to(torch.int64).flatten(-2).unflatten(-1, (-1, 32 // bits))
    words = (code << (bits * torch.arange(32 // bits, device=x.device))).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), s.squeeze(-1), b.squeeze(-1)


def _dequantize(words, s, b, bits):
    """fp32 values [..., D] of packed words."""
    shifts = bits * torch.arange(32 // bits, device=words.device, dtype=torch.int32)
    code = ((words.unsqueeze(-1) >> shifts) & (2 ** bits - 1)).flatten(-2).unflatten(-1, (-1, GROUP))
    return (code.float() * s.unsqueeze(-1).float() + b.unsqueeze(-1).float()).flatten(-2)


def _table(gen, needs, page):
    """A page table of shuffled pages; entries past a request's last page are -1."""
    pages = [-(-max(1, n) // page) for n in needs]
    perm = torch.randperm(sum(pages) + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(needs), max(pages)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, sum(pages) + 3


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


def _empty(n_pages, hk, page, d, bits):
    parts = {}
    for name in ("k", "v"):
        if bits == 16:
            parts[name] = torch.zeros((n_pages, hk, page, d), device="cuda", dtype=torch.bfloat16)
        else:
            parts[name] = torch.zeros((n_pages, hk, page, d * bits // 32), device="cuda", dtype=torch.int32)
            for t in ("_scales", "_biases"):
                parts[name + t] = torch.zeros((n_pages, hk, page, d // GROUP), device="cuda", dtype=torch.float16)
    return parts


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case, "op": case["op"]}
    d = case["d"]

    def bf16(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

    if case["op"] == "rope":
        rows, hq, hk = case["rows"], case["hq"], case["hk"]
        s["qkv"] = bf16(rows, (hq + 2 * hk) * d, scale=1.5)           # the projection's output: q | k | v
        s["qw"], s["kw"] = 1 + bf16(d, scale=0.2), 1 + bf16(d, scale=0.2)
        s["pos"] = (torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
                    + torch.arange(rows, device="cuda")).to(torch.int32)
        half = case["rot"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        if own:
            s["q_out"] = torch.empty((rows, hq * d), dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.empty((rows, hk * d), dtype=torch.bfloat16, device="cuda")
        return s

    page, hk = case["page"], case["hk"]
    if case["op"] == "commit":
        B, n, path = case["batch"], case["rows"], case["path"]
        lens = [(b * 37 + seed) % (2 * page + 1) for b in range(B)]
        s["table"], n_pages = _table(gen, [2 * page + n] * B, page)
        s["k"] = bf16(case["layers"], n_pages, hk, page, d)
        s["v"] = bf16(case["layers"], n_pages, hk, page, d)
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        # half the path is in place already, the rest comes from behind it (a repeated pass finds the same rows)
        keep = path // 2
        far = path + torch.rand((B, n - path), generator=gen, device="cuda").argsort(1)[:, :path - keep].sort(1).values
        s["path"] = torch.cat([torch.arange(keep, device="cuda").expand(B, keep), far], 1).to(torch.int32).contiguous()
        s["path_len"] = torch.full((B,), path, dtype=torch.int32, device="cuda")
        if own:
            s["layers"] = _lib().kv_layers([_lib().kv_cache(s["k"][i], s["v"][i]) for i in range(case["layers"])])
        return s

    counts, lens, bits = _counts(case), _lengths(case), case["bits"]
    offs = _offsets(counts)
    s["table"], n_pages = _table(gen, [n + c for n, c in zip(lens, counts)], page)
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["offs"] = torch.tensor(offs, dtype=torch.int64, device="cuda")
    s["most"] = max(counts)
    rows = offs[-1]
    if case["op"] == "cache":
        qkv = bf16(rows, 6 * hk * d)                                 # q | k | v of a layer with four query heads per key head
        s["new_k"], s["new_v"] = qkv[:, 4 * hk * d:5 * hk * d], qkv[:, 5 * hk * d:]
        s["parts"] = _empty(n_pages, hk, page, d, bits)
    else:
        s["parts"] = _filled(gen, n_pages, hk, page, d, bits)
    if case["op"] == "attend":
        s["q"] = bf16(rows, case["hq"] * d, scale=2.0)
        s["tree"] = _ancestors(gen, counts) if case["tree"] == "tree" else None
    if own:
        lib = _lib()
        s["cache"] = lib.kv_cache(**s["parts"])
        s["row_offsets"] = lib.row_offsets(offs)
        if case["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
            s["workspace"] = lib.workspace(lib.tree_attention_workspace_bytes(s["cache"], s["row_offsets"], case["hq"]))
        else:
            s["out_k"] = torch.empty((rows, hk * d), dtype=torch.bfloat16, device="cuda")
            s["out_v"] = torch.empty_like(s["out_k"])
    return s


# -------------------------------------------------------------- plain forms

def _plain_rope(s):
    c = s["case"]
    rows, hq, hk, d, rot = c["rows"], c["hq"], c["hk"], c["d"], c["rot"]
    turn = torch.remainder(s["pos"].double()[:, None] * s["inv_freq"].double(), 2 * math.pi)
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]

    def one(x, w):
        x = x.unflatten(1, (-1, d)).float()
        if c["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
        r = x[..., :rot]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, x[..., rot:]], -1).flatten(1).to(torch.bfloat16)

    return one(s["qkv"][:, :hq * d], s["qw"]), one(s["qkv"][:, hq * d:(hq + hk) * d], s["kw"])


def _row_places(s, n_rows):
    """Per row: its request, page and place in the page, for rows at kv_len + 0, 1, ..."""
    row = torch.arange(n_rows, device="cuda")
    b = torch.searchsorted(s["offs"], row, right=True) - 1
    pos = s["kv_len"].long()[b] + row - s["offs"][b]
    page = s["case"]["page"]
    return s["table"].long()[b, pos // page], pos % page


def _plain_write(s):
    c = s["case"]
    pg, at = _row_places(s, s["new_k"].shape[0])
    for name in ("k", "v"):
        x = s["new_" + name].unflatten(1, (c["hk"], c["d"]))
        if c["bits"] == 16:
            s["parts"][name][pg, :, at] = x
        else:
            words, scales, biases = _quantize(x.float(), c["bits"])
            s["parts"][name][pg, :, at] = words
            s["parts"][name + "_scales"][pg, :, at] = scales
            s["parts"][name + "_biases"][pg, :, at] = biases


def _plain_values(s, name, at):
    """fp32 cache values at an index of (page, head, place)."""
    p = s["parts"]
    if s["case"]["bits"] == 16:
        return p[name][at].float()
    return _dequantize(p[name][at], p[name + "_scales"][at], p[name + "_biases"][at], s["case"]["bits"])


def _plain_read(s, n_rows):
    pg, at = _row_places(s, n_rows)
    return tuple(_plain_values(s, name, (pg, slice(None), at)).flatten(1).to(torch.bfloat16) for name in ("k", "v"))


def _plain_attend(s):
    c = s["case"]
    hq, hk, d, B, most = c["hq"], c["hk"], c["d"], c["batch"], s["most"]
    pages = s["table"].long().clamp(min=0)
    k, v = (_plain_values(s, name, pages).transpose(1, 2).flatten(2, 3) for name in ("k", "v"))   # [B, hk, T, d]
    row = s["offs"][:-1, None] + torch.arange(most, device="cuda")                                # [B, most]
    real = row < s["offs"][1:, None]
    row = torch.where(real, row, 0)
    q = s["q"][row].float().unflatten(-1, (hk, hq // hk, d)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, hk, most * g, d]
    score = torch.matmul(q, k.transpose(-1, -2)) * (d ** -0.5)
    back = torch.arange(k.shape[2], device="cuda") - s["kv_len"][:, None]                          # place among the drafts
    if s["tree"] is None:
        seen = back[:, None, :] <= torch.arange(most, device="cuda")[:, None]
    else:
        bit = (s["tree"][row][:, :, None] >> back.clamp(0, 63)[:, None, :]) & 1
        seen = (back < 0)[:, None, :] | ((bit == 1) & (back < 64)[:, None, :])
    seen = seen.repeat_interleave(hq // hk, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    o = o.unflatten(2, (most, hq // hk)).permute(0, 2, 1, 3, 4).flatten(2).to(torch.bfloat16)
    return o[real]


def _plain_commit(s):
    page = s["case"]["page"]
    base = s["kv_len"].long()[:, None]
    src, dst = base + s["path"].long(), base + torch.arange(s["path"].shape[1], device="cuda")
    table = s["table"].long()
    from_page, to_page = table.gather(1, src // page), table.gather(1, dst // page)
    for x in (s["k"], s["v"]):
        x[:, to_page, :, dst % page] = x[:, from_page, :, src % page]


def run(s):
    c, op = s["case"], s["op"]
    if op == "rope":
        if not own:
            return _plain_rope(s)
        hq, hk, d = c["hq"], c["hk"], c["d"]
        return _lib().qk_norm_rope(s["qkv"][:, :hq * d], s["qkv"][:, hq * d:(hq + hk) * d], d, s["pos"], s["inv_freq"],
                                   q_weight=s["qw"] if c["norm"] else None, k_weight=s["kw"] if c["norm"] else None, eps=EPS,
                                   norm=c["norm"], interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    if op == "cache":
        if not own:
            _plain_write(s)
            return _plain_read(s, s["new_k"].shape[0])
        _lib().kv_append(s["cache"], s["row_offsets"], s["kv_len"], s["table"], s["new_k"], s["new_v"])
        return _lib().kv_read(s["cache"], s["row_offsets"], s["kv_len"], s["table"], k=s["out_k"], v=s["out_v"])
    if op == "read":
        if not own:
            return _plain_read(s, sum(_counts(c)))
        return _lib().kv_read(s["cache"], s["row_offsets"], s["kv_len"], s["table"], k=s["out_k"], v=s["out_v"])
    if op == "attend":
        if not own:
            return _plain_attend(s)
        return _lib().tree_attention(s["cache"], s["row_offsets"], s["kv_len"], s["table"], s["q"], c["hq"],
                                     tree_mask=s["tree"], out=s["out"], workspace=s["workspace"])
    if not own:
        _plain_commit(s)
    else:
        _lib().kv_commit(s["layers"], s["kv_len"], s["table"], s["path"], s["path_len"])
    return s["k"], s["v"]


# ------------------------------------------------------------- exact values

def _exact_values(words, s, b, bits):
    """fp64 values of int32 code words [..., W], by arithmetic on the words taken as unsigned numbers."""
    u = words.to(torch.int64) % (1 << 32)
    fields = torch.stack([(u // (1 << (bits * j))) % (1 << bits) for j in range(32 // bits)], -1).flatten(-2)
    return fields.double() * s.double().repeat_interleave(GROUP, -1) + b.double().repeat_interleave(GROUP, -1)


def _exact_stored(x, bits):
    """What a cache of `bits` holds for the bf16 rows x [n, heads, d], in fp64 (the format's own roundings applied)."""
    x = x.double()
    if bits == 16:
        return x
    x = x.clamp(-FAR, FAR).reshape(x.shape[0], x.shape[1], -1, GROUP)
    low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    top = 2 ** bits - 1
    scale = ((high - low).float().double() / top).float().half().double()
    bias = low.float().half().double()
    step = ((x - bias).float().double() / torch.where(scale == 0, 1.0, scale)).float().double()
    code = torch.where(scale == 0, 0.0, step.round().clamp(0, top))
    return (code * scale + bias).flatten(-2)


def _exact_sequence(s, name, b, first, count):
    """fp64 [count, hk, d] of request b's positions first .. first + count - 1."""
    c, p = s["case"], s["parts"]
    n = first + count
    pages = s["table"][b, :-(-n // c["page"])].long()
    take = lambda t: t.index_select(0, pages).transpose(1, 2).flatten(0, 1)[first:n]  # noqa: E731
    if c["bits"] == 16:
        return take(p[name]).double()
    return _exact_values(take(p[name]), take(p[name + "_scales"]), take(p[name + "_biases"]), c["bits"])


def exact(case, seed):
    s = prepare(case, seed)
    d = case["d"]
    if case["op"] == "rope":
        rot, half = case["rot"], case["rot"] // 2
        angle = s["pos"].double()[:, None] * s["inv_freq"].double()[None]
        spin = torch.polar(torch.ones_like(angle), angle)[:, None]
        outs = []
        for lo, n, w in ((0, case["hq"], s["qw"]), (case["hq"] * d, case["hk"], s["kw"])):
            x = s["qkv"][:, lo:lo + n * d].double().reshape(-1, n, d)
            if case["norm"]:
                x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
            part = x[..., :rot].reshape(x.shape[0], n, half, 2) if case["interleaved"] else \
                x[..., :rot].reshape(x.shape[0], n, 2, half).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(part.contiguous()) * spin)
            y = y if case["interleaved"] else y.transpose(-1, -2)
            outs.append(torch.cat([y.reshape(x.shape[0], n, rot), x[..., rot:]], -1).reshape(x.shape[0], n * d))
        return tuple(outs)
    if case["op"] == "commit":
        outs = []
        for x in (s["k"], s["v"]):
            y = x.clone()
            for b in range(case["batch"]):
                n, path = int(s["kv_len"][b]), s["path"][b].tolist()
                for j, i in enumerate(path):
                    src, dst = divmod(n + i, case["page"]), divmod(n + j, case["page"])
                    y[:, int(s["table"][b, dst[0]]), :, dst[1]] = x[:, int(s["table"][b, src[0]]), :, src[1]]
            outs.append(y.double())
        return tuple(outs)
    if case["op"] == "cache":
        return tuple(_exact_stored(s["new_" + t].reshape(-1, case["hk"], d), case["bits"]).flatten(1) for t in ("k", "v"))
    counts, lens, offs = _counts(case), _lengths(case), _offsets(_counts(case))
    if case["op"] == "read":
        return tuple(torch.cat([_exact_sequence(s, t, b, lens[b], counts[b]) for b in range(case["batch"])]).flatten(1)
                     for t in ("k", "v"))
    outs = []
    for b in range(case["batch"]):
        n, c = lens[b], counts[b]
        k, v = (_exact_sequence(s, t, b, 0, n + c).repeat_interleave(case["hq"] // case["hk"], 1) for t in ("k", "v"))
        q = s["q"][offs[b]:offs[b + 1]].double().reshape(c, case["hq"], d)
        hide = torch.zeros((c, n + c), dtype=torch.bool)
        for i in range(c):
            bits = (int(s["tree"][offs[b] + i]) if s["tree"] is not None else (1 << (i + 1)) - 1)
            hide[i, n:] = torch.tensor([not bits >> j & 1 for j in range(c)])
        z = torch.einsum("chd,thd->hct", q, k) / math.sqrt(d)
        z = z.masked_fill(hide.cuda()[None], -math.inf)
        outs.append(torch.einsum("hct,thd->chd", (z - z.logsumexp(-1, keepdim=True)).exp(), v).reshape(c, -1))
    return torch.cat(outs)
