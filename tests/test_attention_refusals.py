"""The attention-side calls reject bad arguments on the host, before any launch (no GPU needed)."""

import ctypes

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from speculative_decoding_verify_qmm_gb300.binding import SV_EINVAL, SV_EUNSUPPORTED, SV_OK

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


def _cache(**kw):
    f = dict(k=256, v=512, k_scales=256, k_biases=256, v_scales=256, v_biases=256, n_pages=8, page_size=16,
             n_kv_heads=2, head_dim=64, bits=8)
    f.update(kw)
    return binding.KVCacheView(*[f[n] for n, _ in binding.KVCacheView._fields_])


def _offs(*v):
    return (ctypes.c_int32 * len(v))(*v)


def _rope(raw, q=16, ldq=256, k=16, ldk=128, rows=2, hq=4, hk=2, d=64, norm=1, qw=None, kw=None, eps=1e-6, pos=16,
          inv=16, rot=64, inter=0, qo=32, ldqo=256, ko=32, ldko=128):
    return raw.sv_qk_norm_rope(q, ldq, k, ldk, rows, hq, hk, d, norm, qw, kw, eps, pos, inv, rot, inter, qo, ldqo, ko,
                               ldko, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), SV_EINVAL), (dict(k=None), SV_EINVAL), (dict(qo=None), SV_EINVAL), (dict(ko=None), SV_EINVAL),
    (dict(q=17), SV_EINVAL), (dict(rows=-1), SV_EINVAL), (dict(rows=(1 << 20) + 1), SV_EINVAL), (dict(hq=0), SV_EINVAL),
    (dict(hk=-1), SV_EINVAL), (dict(d=60), SV_EUNSUPPORTED), (dict(d=264), SV_EUNSUPPORTED),
    (dict(rot=8), SV_EUNSUPPORTED), (dict(rot=80), SV_EUNSUPPORTED), (dict(rot=-16), SV_EUNSUPPORTED),
    (dict(ldq=255), SV_EINVAL), (dict(ldko=64), SV_EINVAL), (dict(eps=-1.0), SV_EINVAL),
    (dict(eps=float("nan")), SV_EINVAL), (dict(pos=None), SV_EINVAL), (dict(inv=None), SV_EINVAL),
    (dict(qo=16, ldqo=264), SV_EINVAL), (dict(pos=18), SV_EINVAL), (dict(qw=33), SV_EINVAL)])
def test_norm_rope_refuses(raw, bad, status):
    assert _rope(raw, **bad) == status
    assert raw.sv_last_error()


def test_norm_rope_without_rows_is_done(raw):
    assert _rope(raw, rows=0) == SV_OK
    assert _rope(raw, rows=0, hk=0, k=None, ko=None, rot=0, pos=None, inv=None) == SV_OK


CACHE_BAD = [
    (dict(bits=2), SV_EUNSUPPORTED), (dict(bits=5), SV_EUNSUPPORTED), (dict(head_dim=96), SV_EUNSUPPORTED),
    (dict(head_dim=0), SV_EUNSUPPORTED), (dict(head_dim=320), SV_EUNSUPPORTED), (dict(page_size=8), SV_EUNSUPPORTED),
    (dict(page_size=48), SV_EUNSUPPORTED), (dict(page_size=1 << 17), SV_EUNSUPPORTED), (dict(n_kv_heads=0), SV_EINVAL),
    (dict(n_kv_heads=257), SV_EINVAL), (dict(n_pages=0), SV_EINVAL), (dict(k=None), SV_EINVAL), (dict(v=None), SV_EINVAL),
    (dict(k=264), SV_EINVAL), (dict(v=256), SV_EINVAL), (dict(v_biases=None), SV_EINVAL), (dict(k_scales=258), SV_EINVAL)]


def _append(raw, cache, B=1, offs=None, lens=16, table=16, pages=4, k=16, ldk=128, v=16, ldv=128, read=False):
    call = raw.sv_kv_read if read else raw.sv_kv_append
    ref = ctypes.byref(cache) if cache is not None else None
    return call(ref, B, offs if offs is not None else _offs(0, 3), lens, table, pages, k, ldk, v, ldv, None)


@pytest.mark.parametrize("read", [False, True])
def test_append_and_read_refuse(raw, read):
    for bad, status in CACHE_BAD:
        assert _append(raw, _cache(**bad), read=read) == status, bad
    assert _append(raw, None, read=read) == SV_EINVAL
    ok = _cache()
    for bad, status in [(dict(B=0), SV_EINVAL), (dict(B=257), SV_EINVAL), (dict(offs=_offs(1, 3)), SV_EINVAL),
                        (dict(B=2, offs=_offs(0, 3, 2)), SV_EINVAL), (dict(lens=None), SV_EINVAL), (dict(lens=18), SV_EINVAL),
                        (dict(table=None), SV_EINVAL), (dict(pages=0), SV_EINVAL), (dict(pages=(1 << 26) + 1), SV_EUNSUPPORTED),
                        (dict(k=None), SV_EINVAL), (dict(v=None), SV_EINVAL), (dict(k=17), SV_EINVAL),
                        (dict(ldk=127), SV_EINVAL), (dict(ldv=127), SV_EINVAL),
                        (dict(offs=_offs(0, (1 << 22) + 1)), SV_EUNSUPPORTED)]:
        assert _append(raw, ok, read=read, **bad) == status, bad
    assert _append(raw, ok, offs=_offs(0, 0), read=read) == SV_OK


def _attend(raw, cache, B=1, offs=None, lens=16, table=16, pages=4, q=16, ldq=256, hq=4, scale=0.1, mask=None, out=16,
            ldo=256, ws=256, ws_bytes=1 << 30):
    ref = ctypes.byref(cache) if cache is not None else None
    return raw.sv_tree_attention(ref, B, offs if offs is not None else _offs(0, 3), lens, table, pages, q, ldq, hq, scale,
                                 mask, out, ldo, ws, ws_bytes, None)


def test_tree_attention_refuses(raw):
    for bad, status in CACHE_BAD:
        assert _attend(raw, _cache(**bad)) == status, bad
    ok = _cache()
    for bad, status in [(dict(B=0), SV_EINVAL), (dict(offs=_offs(0, 65)), SV_EUNSUPPORTED), (dict(offs=_offs(2, 3)), SV_EINVAL),
                        (dict(lens=None), SV_EINVAL), (dict(table=None), SV_EINVAL), (dict(pages=0), SV_EINVAL),
                        (dict(q=None), SV_EINVAL), (dict(out=None), SV_EINVAL), (dict(q=24), SV_EINVAL),
                        (dict(ldq=260), SV_EINVAL), (dict(ldq=248), SV_EINVAL), (dict(ldo=248), SV_EINVAL),
                        (dict(hq=3), SV_EINVAL), (dict(hq=0), SV_EINVAL), (dict(hq=130, ldq=1 << 14, ldo=1 << 14), SV_EINVAL),
                        (dict(scale=float("inf")), SV_EINVAL), (dict(scale=float("nan")), SV_EINVAL),
                        (dict(mask=20), SV_EINVAL), (dict(ws=None), SV_EINVAL), (dict(ws=128), SV_EINVAL),
                        (dict(ws_bytes=0), SV_EINVAL)]:
        assert _attend(raw, ok, **bad) == status, bad
    assert _attend(raw, _cache(head_dim=192), ldq=1024, ldo=1024) == SV_EUNSUPPORTED
    assert _attend(raw, ok, pages=1, offs=_offs(0, ok.page_size + 1)) == SV_EINVAL    # more rows than the table has places
    assert raw.sv_tree_attention_workspace_bytes(ctypes.byref(ok), 1, _offs(0, 65), 4) == 0
    assert raw.sv_tree_attention_workspace_bytes(None, 1, _offs(0, 1), 4) == 0


def test_commit_refuses(raw):
    def call(layers=None, n=1, B=1, lens=16, table=16, pages=4, path=16, most=8, plen=16):
        layers = (binding.KVCacheView * 2)(_cache(), _cache()) if layers is None else layers
        return raw.sv_kv_commit(layers, n, B, lens, table, pages, path, most, plen, None)
    for bad, status in CACHE_BAD:
        assert call((binding.KVCacheView * 2)(_cache(), _cache(**bad)), n=2) == status, bad
    for bad, status in [(dict(n=0), SV_EINVAL), (dict(n=1025), SV_EINVAL), (dict(B=0), SV_EINVAL), (dict(B=257), SV_EINVAL),
                        (dict(lens=None), SV_EINVAL), (dict(table=None), SV_EINVAL), (dict(pages=0), SV_EINVAL),
                        (dict(path=None), SV_EINVAL), (dict(plen=None), SV_EINVAL), (dict(most=0), SV_EINVAL),
                        (dict(most=65), SV_EINVAL), (dict(path=18), SV_EINVAL)]:
        assert call(**bad) == status, bad
    assert call((binding.KVCacheView * 2)(_cache(), _cache(n_pages=9)), n=2) == SV_EINVAL
    assert call((binding.KVCacheView * 2)(_cache(), _cache(bits=4)), n=2) == SV_EINVAL
    assert call((binding.KVCacheView * 2)(_cache(), _cache()), n=2) == SV_EINVAL          # the same memory twice
    assert call((binding.KVCacheView * 2)(_cache(), _cache(k=1024, v=256)), n=2) == SV_EINVAL
    assert raw.sv_kv_commit(None, 1, 1, 16, 16, 4, 16, 8, 16, None) == SV_EINVAL


def test_binding_refuses_host_tensors():
    import torch
    build.build()
    lib = binding.load()
    x = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(binding.SVError):
        lib.kv_cache(x, x)
    with pytest.raises(binding.SVError):
        lib.kv_layers([])
