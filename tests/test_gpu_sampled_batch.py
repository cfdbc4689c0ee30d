"""Samples of one prompt, served together: fork, then rounds of reserve, append, attention over the shared prefix, accept, commit and
trim, some of them replayed from a graph, then half of the samples freed and the cache compacted.  Beside it the host keeps every
sample's sequence; caches are compared exactly, attention with its fp64 bound, decisions with the oracle's."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests.test_gpu_attention import bf16, i32, offsets
from tests.test_gpu_attention_shared import Batch

pytestmark = pytest.mark.gpu

LAYERS, PAGE, HQ, HK, D, V, T = 2, 16, 16, 8, 64, 500, 0.8
N, ROWS, PROMPT, SLOTS = 12, 9, 6005, 14


def tree(r, q):
    """A random tree of ROWS nodes with children drawn from q without replacement: parents, tokens, masks."""
    parent, token, masks = [-1], [0], [1]
    kids = [[] for _ in range(ROWS)]
    for i in range(1, ROWS):
        v = int(r.integers(max(0, i - 4), i))
        p = q[v].astype(np.float64)
        p[kids[v]] = 0
        x = int(r.choice(V, p=p / p.sum()))
        kids[v].append(x)
        parent.append(v)
        token.append(x)
        masks.append(masks[v] | 1 << i)
    return parent, token, masks


@pytest.mark.parametrize("bits", [16, 8])
def test_rounds_of_forked_samples(lib, bits):
    r = np.random.default_rng(bits)
    width, n_pages = (PROMPT + 200) // PAGE + 1, PROMPT // PAGE + 1 + SLOTS * 12
    pool = lib.kv_pages_alloc(n_pages, PAGE, SLOTS, width)
    caches = lib.kv_layers([lib.kv_cache_alloc(n_pages, PAGE, HK, D, bits) for _ in range(LAYERS)])
    ws = torch.zeros(lib.kv_reserve_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    counts, copies = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros((SLOTS, 3), dtype=torch.int32, device="cuda")
    # the prompt goes to slot 0, the samples are slots 1 .. N (slot N + 1 stays empty)
    lib.kv_reserve(pool, caches, i32([0] * SLOTS), i32([PROMPT] + [-1] * (SLOTS - 1)), counts, copies, ws)
    rows = [[bf16(r, PROMPT, HK * D) for _ in "kv"] for _ in range(LAYERS)]
    for cache, (k, v) in zip(caches.caches, rows):
        lib.kv_append(cache, [0, PROMPT], i32([0]), pool.block_table, k.cuda(), v.cuda())
    lib.kv_fork(pool, i32([0] * N), i32(list(range(1, N + 1))), i32([PROMPT] * N))
    seqs = [[[k, v] for k, v in rows] for _ in range(N)]
    lens = [PROMPT] * N

    offs = offsets([ROWS] * N)
    groups = lib.prefix_groups([0, N], [PROMPT // PAGE])
    kv_len = torch.zeros(SLOTS, dtype=torch.int32, device="cuda")
    kv_len[0:N + 1] = PROMPT
    sampled = torch.zeros(SLOTS, dtype=torch.bool, device="cuda")
    sampled[1:N + 1] = True
    M, table, mine = N * ROWS, pool.block_table[1:N + 1], kv_len[1:N + 1]
    dev = dict(k=torch.zeros((LAYERS, M, HK * D), dtype=torch.bfloat16, device="cuda"), q=torch.zeros((LAYERS, M, HQ * D), dtype=torch.bfloat16, device="cuda"),
               mask=torch.zeros(M, dtype=torch.int64, device="cuda"), z=torch.zeros((M, V), device="cuda"), qd=torch.zeros((M, V), device="cuda"),
               parent=i32([0] * M), token=i32([0] * M), u=torch.zeros(M, device="cuda"))
    dev["v"] = torch.zeros_like(dev["k"])
    att = torch.zeros((LAYERS, M, HQ * D), dtype=torch.bfloat16, device="cuda")
    out = (i32([0] * N), i32([-1] * M), torch.full((N, ROWS), -1, dtype=torch.int32, device="cuda"))
    minus = torch.full_like(kv_len, -1)
    trimmed, scratch = torch.zeros_like(counts), torch.zeros(
        lib.tree_attention_shared_workspace_bytes(caches.caches[0], groups, offs, HQ), dtype=torch.uint8, device="cuda")

    def one_round():
        lib.kv_reserve(pool, caches, kv_len, torch.where(sampled, kv_len + ROWS, minus), counts, copies, ws)
        for l, cache in enumerate(caches.caches):
            lib.kv_append(cache, offs, mine, table, dev["k"][l], dev["v"][l])
            lib.tree_attention_shared(cache, groups, offs, mine, table, dev["q"][l], HQ, tree_mask=dev["mask"], out=att[l], workspace=scratch)
        for t in out[1:]:
            t.fill_(-1)
        lib.tree_accept(offs, dev["z"], dev["parent"], dev["token"], T, q=dev["qd"], u=dev["u"], distinct=True, out=out)
        lib.kv_commit(caches, mine, table, out[2], out[0])
        kv_len[1:N + 1] += out[0]
        lib.kv_reserve(pool, caches, kv_len, torch.where(sampled, kv_len, minus), trimmed, copies, ws)

    def feed():
        draft = r.standard_normal((M, V)).astype(np.float32)
        z = (draft + 0.5 * r.standard_normal((M, V))).astype(np.float32) * 2
        w = np.exp(draft.astype(np.float64) * 2 / T)
        host = dict(k=torch.stack([bf16(r, M, HK * D) for _ in range(LAYERS)]), v=torch.stack([bf16(r, M, HK * D) for _ in range(LAYERS)]),
                    q=torch.stack([bf16(r, M, HQ * D, scale=1.5) for _ in range(LAYERS)]), z=torch.from_numpy(z),
                    qd=torch.from_numpy((w / w.sum(1, keepdims=True)).astype(np.float32)), u=torch.from_numpy(r.random(M).astype(np.float32)))
        trees = [tree(r, host["qd"][offs[b]:offs[b + 1]].numpy()) for b in range(N)]
        host["parent"], host["token"], masks = (sum((t[i] for t in trees), []) for i in range(3))
        for name in ("parent", "token"):
            host[name] = torch.tensor(host[name], dtype=torch.int32)
        host["mask"] = torch.tensor(masks, dtype=torch.int64)
        for name, t in host.items():
            dev[name].copy_(t)
        return host, masks

    def reference(extra=None):
        """Fresh caches of the sequences (and the drafts behind them), each sample with pages of its own."""
        total = [lens[b] + (ROWS if extra else 0) for b in range(N)]
        per = [-(-n // PAGE) for n in total]
        tab = np.zeros((N, max(per)), np.int32)
        for b in range(N):
            tab[b, :per[b]] = np.arange(sum(per[:b]), sum(per[:b + 1]))
        made = []
        for l in range(LAYERS):
            c = lib.kv_cache_alloc(sum(per), PAGE, HK, D, bits)
            for b in range(N):
                k, v = (torch.cat([seqs[b][l][i]] + ([extra["kv"[i]][l][offs[b]:offs[b + 1]]] if extra else [])).cuda() for i in range(2))
                lib.kv_append(c, [0, total[b]], i32([0]), i32(tab[b:b + 1].tolist()), k, v)
            made.append(c)
        return made, tab

    def caches_hold_the_sequences(samples):
        made, tab = reference()
        for l in range(LAYERS):
            for b in samples:
                got = lib.kv_read(caches.caches[l], [0, lens[b]], i32([0]), pool.block_table[b + 1:b + 2])
                want = lib.kv_read(made[l], [0, lens[b]], i32([0]), i32(tab[b:b + 1].tolist()))
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    graph = None
    for step in range(5):
        host, masks = feed()
        if step == 2:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one_round()
        one_round() if graph is None else graph.replay()
        torch.cuda.synchronize()
        assert lib.device_error() == 0 and counts[0].item() == 0 and trimmed.tolist() == [0, 0, 0]
        made, tab = reference(host)
        for l in range(LAYERS):
            case = SimpleNamespace(d=D, hq=HQ, hk=HK, bits=bits, counts=[ROWS] * N, lens=lens, offs=offs, table=tab, page=PAGE, cache=made[l],
                                   masks=masks, q=host["q"][l])
            Batch.check(case, att[l], requests=[0, step + 1, N - 1])
        length, tokens, path = (t.cpu().numpy() for t in out)
        for b in range(N):
            s = slice(offs[b], offs[b + 1])
            want, emitted, margin = ot.accept(host["z"][s].numpy(), host["parent"][s].tolist(), host["token"][s].tolist(), T, host["qd"][s].numpy(),
                                              host["u"][s].numpy(), True, max_path=ROWS)
            assert margin < 0 or (path[b, :length[b]].tolist() == want and tokens[s][:length[b]].tolist() == emitted)
            for l in range(LAYERS):
                for i in range(2):
                    seqs[b][l][i] = torch.cat([seqs[b][l][i], host["kv"[i]][l][s][torch.from_numpy(path[b, :length[b]].astype(np.int64))]])
            lens[b] += int(length[b])
        assert kv_len[1:N + 1].tolist() == lens and pool.held[1:N + 1].tolist() == [-(-n // PAGE) for n in lens]
        caches_hold_the_sequences(range(N) if step in (0, 4) else [step])
    # the prompt's own slot and half of the samples go; what is left moves to the front
    keep = kv_len.clone()
    keep[0] = 0
    keep[2:N + 1:2] = 0
    need = torch.where((keep == 0) & (pool.held > 0), 0, -1).to(torch.int32)
    lib.kv_reserve(pool, caches, keep, need, counts, copies, ws)
    live, moves = lib.kv_compact(pool, caches)
    left = [b for b in range(N) if b % 2 == 0]
    assert lib.device_error() == 0 and live[0].item() == PROMPT // PAGE + sum(-(-lens[b] // PAGE) - PROMPT // PAGE for b in left)
    assert pool.refs[:PROMPT // PAGE].max().item() == len(left) and not pool.refs[live[0].item():].any()
    caches_hold_the_sequences(left)
