"""Tree accept, attention over shared prefixes and the pages of a cache refuse bad arguments on the host, before any launch."""

import ctypes

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from speculative_decoding_verify_qmm_gb300.binding import SV_EINVAL, SV_EUNSUPPORTED, SV_OK
from tests.test_attention_refusals import CACHE_BAD, _cache, _offs


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


def _accept(raw, B=1, offs=None, logits=16, ldl=100, top=None, total=None, arg=None, parent=16, token=16, q=16, ldq=100, distinct=0, V=100, T=0.5,
            u=16, top_k=0, top_p=1.0, n=16, tokens=16, path=16, most=8):
    return raw.sv_tree_accept(B, offs if offs is not None else _offs(0, 3), logits, ldl, top, total, arg, parent, token, q, ldq, distinct, V, T, u,
                              top_k, top_p, n, tokens, path, most, None, 0, None)


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), SV_EINVAL), (dict(B=257), SV_EINVAL), (dict(offs=_offs(1, 3)), SV_EINVAL), (dict(offs=_offs(0, 0)), SV_EINVAL),
    (dict(B=2, offs=_offs(0, 3, 3)), SV_EINVAL), (dict(B=2, offs=_offs(0, 3, 2)), SV_EINVAL), (dict(offs=_offs(0, 65)), SV_EUNSUPPORTED),
    (dict(V=1), SV_EINVAL), (dict(V=(1 << 22) + 1, ldl=1 << 23, ldq=1 << 23), SV_EINVAL), (dict(ldl=99), SV_EINVAL), (dict(ldq=99), SV_EINVAL),
    (dict(T=-0.1), SV_EINVAL), (dict(T=2.0 ** 121), SV_EINVAL), (dict(T=float("inf")), SV_EINVAL), (dict(T=float("nan")), SV_EINVAL), (dict(u=None), SV_EINVAL),
    (dict(logits=None), SV_EINVAL), (dict(parent=None), SV_EINVAL), (dict(token=None), SV_EINVAL), (dict(n=None), SV_EINVAL),
    (dict(tokens=None), SV_EINVAL), (dict(path=None), SV_EINVAL), (dict(logits=18), SV_EINVAL), (dict(q=17), SV_EINVAL), (dict(u=18), SV_EINVAL),
    (dict(path=18), SV_EINVAL), (dict(top=16), SV_EINVAL), (dict(top=16, arg=16), SV_EINVAL), (dict(total=16, arg=16), SV_EINVAL),
    (dict(T=0.0, top=16), SV_EINVAL), (dict(top_k=-1), SV_EINVAL), (dict(top_p=0.0), SV_EINVAL), (dict(top_p=1.1), SV_EINVAL),
    (dict(top_p=float("nan")), SV_EINVAL), (dict(most=0), SV_EINVAL), (dict(most=65), SV_EINVAL)])
def test_tree_accept_refuses(raw, bad, status):
    assert _accept(raw, **bad) == status
    assert raw.sv_last_error()
    assert raw.sv_tree_accept_workspace_bytes(64) == 0


def _shared(raw, cache, G=1, goffs=None, pages=None, B=2, offs=None, lens=16, table=16, width=4, q=16, ldq=256, hq=4, scale=0.1, mask=None, out=16,
            ldo=256, ws=256, ws_bytes=1 << 40):
    goffs, pages = goffs if goffs is not None else _offs(0, 2), pages if pages is not None else _offs(2)
    offs = offs if offs is not None else _offs(0, 3, 5)
    ref = ctypes.byref(cache) if cache is not None else None
    size = raw.sv_tree_attention_shared_workspace_bytes(ref, G, goffs, pages, B, offs, hq)
    st = raw.sv_tree_attention_shared(ref, G, goffs, pages, B, offs, lens, table, width, q, ldq, hq, scale, mask, out, ldo, ws, ws_bytes, None)
    return st, size


def test_tree_attention_shared_refuses(raw):
    for bad, status in CACHE_BAD:
        assert _shared(raw, _cache(**bad)) == (status, 0), bad
    assert _shared(raw, None) == (SV_EINVAL, 0)
    ok = _cache()
    for bad, status in [(dict(G=0), SV_EINVAL), (dict(G=257), SV_EINVAL), (dict(goffs=_offs(1, 2)), SV_EINVAL), (dict(goffs=_offs(0, 3)), SV_EINVAL),
                        (dict(G=2, goffs=_offs(0, 3, 2), pages=_offs(1, 1)), SV_EINVAL), (dict(G=2, goffs=_offs(0, -1, 2), pages=_offs(1, 1)), SV_EINVAL),
                        (dict(pages=_offs(-1)), SV_EINVAL), (dict(pages=_offs((1 << 26) + 1)), SV_EINVAL), (dict(pages=_offs(2 ** 31 - 1)), SV_EINVAL),
                        (dict(B=0), SV_EINVAL), (dict(offs=_offs(0, 65, 66)), SV_EUNSUPPORTED), (dict(offs=_offs(0, 3, 2)), SV_EINVAL), (dict(hq=3), SV_EINVAL)]:
        assert _shared(raw, ok, **bad) == (status, 0), bad
    for bad, status in [(dict(lens=None), SV_EINVAL), (dict(table=None), SV_EINVAL), (dict(width=0), SV_EINVAL), (dict(q=None), SV_EINVAL),
                        (dict(out=None), SV_EINVAL), (dict(q=24), SV_EINVAL), (dict(ldq=260), SV_EINVAL), (dict(ldo=248), SV_EINVAL),
                        (dict(scale=float("nan")), SV_EINVAL), (dict(scale=3e38), SV_EINVAL), (dict(mask=20), SV_EINVAL), (dict(ws=None), SV_EINVAL),
                        (dict(ws=128), SV_EINVAL), (dict(ws_bytes=0), SV_EINVAL), (dict(pages=_offs(5)), SV_EINVAL), (dict(q=4096, out=4096, ldo=264), SV_EINVAL)]:
        assert _shared(raw, ok, **bad)[0] == status, bad
    assert _shared(raw, _cache(head_dim=192), ldq=1024, ldo=1024)[0] == SV_EUNSUPPORTED
    # a prefix that leaves the tables no place for a request's rows, where it is shared
    wide = dict(B=64, offs=_offs(*range(0, 193, 3)), goffs=_offs(0, 64), width=1024, pages=_offs(1024))
    assert _shared(raw, _cache(n_kv_heads=8, n_pages=4096), hq=8, ldq=512, ldo=512, **wide)[0] == SV_EINVAL
    assert b"places" in raw.sv_last_error()


def _pool(**kw):
    f = dict(refs=16, block_table=16, held=16, n_pages=8, page_size=16, slots=4, table_pages=6)
    f.update(kw)
    return binding.KVPagesView(*[f[n] for n, _ in binding.KVPagesView._fields_])


POOL_BAD = [(dict(refs=None), SV_EINVAL), (dict(block_table=None), SV_EINVAL), (dict(held=None), SV_EINVAL), (dict(refs=18), SV_EINVAL),
            (dict(held=17), SV_EINVAL), (dict(n_pages=0), SV_EINVAL), (dict(n_pages=(1 << 30) + 1), SV_EINVAL), (dict(page_size=8), SV_EUNSUPPORTED),
            (dict(page_size=24), SV_EUNSUPPORTED), (dict(page_size=1 << 17), SV_EUNSUPPORTED), (dict(slots=0), SV_EINVAL), (dict(slots=257), SV_EINVAL),
            (dict(table_pages=0), SV_EINVAL), (dict(table_pages=(1 << 26) + 1), SV_EUNSUPPORTED)]


def _layers(*caches):
    return (binding.KVCacheView * len(caches))(*caches)


def test_page_calls_refuse(raw):
    def fork(pool, n=1, parent=16, child=16, tokens=16):
        return raw.sv_kv_fork(None if pool is None else ctypes.byref(pool), n, parent, child, tokens, None)

    def reserve(pool, layers=None, n=1, keep=16, need=16, counts=16, copies=16, ws=256, ws_bytes=1 << 20):
        return raw.sv_kv_reserve(None if pool is None else ctypes.byref(pool), _layers(_cache()) if layers is None else layers, n, keep, need, counts,
                                 copies, ws, ws_bytes, None)

    def compact(pool, layers=None, n=1, counts=16, moves=16):
        return raw.sv_kv_compact(None if pool is None else ctypes.byref(pool), _layers(_cache()) if layers is None else layers, n, counts, moves, None)
    for bad, status in POOL_BAD:
        assert fork(_pool(**bad)) == reserve(_pool(**bad)) == compact(_pool(**bad)) == status, bad
        assert raw.sv_kv_reserve_workspace_bytes(ctypes.byref(_pool(**bad))) == 0
    assert fork(None) == reserve(None) == compact(None) == SV_EINVAL and raw.sv_kv_reserve_workspace_bytes(None) == 0
    for bad in (dict(n=-1), dict(n=257), dict(parent=None), dict(child=None), dict(tokens=None), dict(parent=18)):
        assert fork(_pool(), **bad) == SV_EINVAL, bad
    assert fork(_pool(), n=0, parent=None, child=None, tokens=None) == SV_OK
    for call in (reserve, compact):
        for bad, status in CACHE_BAD:
            assert call(_pool(), layers=_layers(_cache(k=4096, v=8192), _cache(**bad)), n=2) == status, bad
        for layers in ((_cache(), _cache()), (_cache(), _cache(k=4096, v=256)), (_cache(), _cache(k=4096, v=8192, bits=4)),
                       (_cache(), _cache(k=4096, v=8192, n_pages=9)), (_cache(), _cache(k=4096, v=8192, head_dim=128))):
            assert call(_pool(), layers=_layers(*layers), n=2) == SV_EINVAL
        assert call(_pool(), n=-1) == call(_pool(), n=1025) == call(_pool(n_pages=9)) == call(_pool(page_size=32)) == call(_pool(), counts=None) == SV_EINVAL
    for bad in (dict(keep=None), dict(need=None), dict(copies=None), dict(keep=18), dict(ws=None), dict(ws=128), dict(ws_bytes=0)):
        assert reserve(_pool(), **bad) == SV_EINVAL, bad
    assert compact(_pool(), moves=None) == compact(_pool(), moves=18) == SV_EINVAL
    assert raw.sv_kv_reserve(ctypes.byref(_pool()), None, 1, 16, 16, 16, 16, 256, 1 << 20, None) == SV_EINVAL


def test_copy_pages_refuses(raw):
    a, b, c = _cache(), _cache(k=4096, v=8192, n_pages=20), _cache(k=16384, v=32768)

    def call(src=None, dst=None, n_layers=1, n=1, at=16, to=16):
        return raw.sv_kv_copy_pages(_layers(a) if src is None else src, _layers(b) if dst is None else dst, n_layers, n, at, to, None)
    for bad, status in CACHE_BAD:
        assert call(src=_layers(_cache(**bad)), dst=_layers(_cache(**bad))) == status, bad
    for bad in (dict(n_layers=0), dict(n_layers=1025), dict(n=-1), dict(n=(1 << 24) + 1), dict(at=None), dict(to=None), dict(at=18),
                dict(dst=_layers(_cache(k=4096, v=8192, bits=4))), dict(dst=_layers(_cache(k=4096, v=8192, page_size=32))),
                dict(src=_layers(a, c), dst=_layers(b, b), n_layers=2),                                   # one cache written twice
                dict(src=_layers(a, c), dst=_layers(c, a), n_layers=2)):                                  # a layer's source is another's destination
        assert call(**bad) == SV_EINVAL, bad
    assert call(n=0, at=None, to=None) == SV_OK
    assert raw.sv_kv_copy_pages(None, None, 1, 1, 16, 16, None) == SV_EINVAL


def test_binding_refuses():
    import torch
    build.build()
    lib = binding.load()
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)                                                   # noqa: E731
    with pytest.raises(binding.SVError):
        lib.kv_pages(ints(4), ints(2, 3), ints(2), 16)                                                    # host tensors
    for offs, pages in (([0, 2], [1, 2]), ([0], []), ([0, 2 ** 31], [1]), ([0, 2], [2 ** 31])):
        if len(offs) == len(pages) + 1 and not pages:
            assert lib.prefix_groups(offs, pages).n == 0                                                  # (the call refuses it)
            continue
        with pytest.raises(binding.SVError):
            lib.prefix_groups(offs, pages)
    z = torch.zeros((3, 10))
    with pytest.raises(binding.SVError, match="current device"):
        lib.tree_accept([0, 3], z, ints(3), ints(3), 0.0)
    for offs in ([0, 2 ** 32 + 2], [0, 3, 0], []):
        with pytest.raises(binding.SVError, match="row_offsets"):
            lib.tree_accept(offs, z, ints(3), ints(3), 0.0)
    k = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    cache = binding.KVCache(binding.KVCacheView(k.data_ptr(), k.data_ptr(), None, None, None, None, 2, 16, 2, 64, 16), [k, k])
    pool = binding.KVPages(binding.KVPagesView(256, 256, 256, 2, 16, 2, 4), ints(2), ints(2, 4), ints(2))
    for call in (lambda: lib.kv_fork(pool, ints(1), ints(1), ints(1)), lambda: lib.kv_reserve(pool, [cache], ints(2), ints(2)),
                 lambda: lib.kv_compact(pool, None), lambda: lib.kv_copy_pages([cache], ints(1), ints(1)),
                 lambda: lib.kv_fork(pool, ints(1), ints(2), ints(1)), lambda: lib.kv_copy_pages([cache], ints(1), ints(2))):
        with pytest.raises(binding.SVError):
            call()
