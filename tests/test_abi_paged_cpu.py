"""Host rules of the paged-cache entry points (no GPU work: every call here is
refused, or has nothing to do)."""

import ctypes

import pytest

from helpers import ensure_built


@pytest.fixture(scope="module")
def lib():
    ensure_built()
    from kv_cache_eviction_snapkv_gb300 import _native
    return _native.lib()


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)


def pool(**kw):
    from kv_cache_eviction_snapkv_gb300 import _native
    d = dict(num_layers=2, num_pages=10, page_size=16, num_kv_heads=2, head_dim=128, dtype=0,
             layer_stride=0, page_stride=0, K=4096, V=8192)
    d.update(kw)
    return _native.KvselPages(**d)


def rows(data=4096, layer=0, token=1024):
    from kv_cache_eviction_snapkv_gb300 import _native
    return ctypes.byref(_native.KvselRows(data, layer, token))


def attention(lib, p, S=3, H=4, q=P, table=P, width=5, lens=P, out=P, ws=P, ws_bytes=1 << 40):
    return lib.kvsel_paged_attention(ctypes.byref(p), S, H, q, table, width, lens, out, None, ws,
                                     ws_bytes, None)


def append(lib, p, n=3, H=4, q=True, k=True, v=True, rope=None, w=None, eps=1e-6, pos=P, S=3,
           table=P, width=5, seqs=P, cache_pos=P, q_out=P):
    r = None
    if rope is not None:
        from kv_cache_eviction_snapkv_gb300 import _native
        r = ctypes.byref(_native.KvselRope(rope, 0, 4096, 1.0))
    return lib.kvsel_paged_append(ctypes.byref(p), n, H, rows() if q is True else q,
                                  rows() if k is True else k, rows() if v is True else v, r, w, w, eps,
                                  pos, S, table, width, seqs, cache_pos, q_out, None)


def compact(lib, p, S=3, table=P, width=5, lens=P, idx=P, rows_=20, offs=P, most=8):
    return lib.kvsel_paged_compact(ctypes.byref(p), S, table, width, lens, idx, rows_, offs, most,
                                   None, None, None)


def update(lib, p, n_in=3, table=P, width=5, lens=P, n_out=3, parents=P, new=P,
           out=ctypes.c_void_p(1 << 20), ref=P, ws=P, ws_bytes=1 << 30):
    return lib.kvsel_pages_update(ctypes.byref(p), n_in, table, width, lens, n_out, parents, new, out,
                                  ref, None, ws, ws_bytes, None)


BAD_POOLS = [
    (dict(num_layers=0), 1), (dict(num_pages=-1), 1), (dict(page_size=0), 1), (dict(num_kv_heads=0), 1),
    (dict(head_dim=0), 1), (dict(dtype=2), 1), (dict(layer_stride=-16), 1), (dict(page_stride=1024), 1),
    (dict(page_stride=4096 + 8), 1), (dict(layer_stride=4096 * 10 + 8), 1), (dict(K=4096 + 16), 1),
    (dict(V=None), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2), (dict(page_size=24), 2),
    (dict(num_pages=1 << 28), 2), (dict(num_pages=1 << 26, num_kv_heads=64), 2),
    (dict(num_kv_heads=1 << 30), 2), (dict(page_stride=1 << 50), 2), (dict(layer_stride=1 << 60), 2),
]


@pytest.mark.parametrize("change,status", BAD_POOLS)
def test_pool_rules_hold_for_every_call(lib, change, status):
    p = pool(**change)
    assert attention(lib, p, H=p.num_kv_heads if 0 < p.num_kv_heads < 100 else 4) == status
    assert append(lib, p) == status
    assert compact(lib, p) == status
    assert update(lib, p) == status


def test_tables_of_too_many_rows(lib):
    """2^30 rows a sequence, whatever the page size."""
    for ps, width in ((1, 1 << 30), (16, 1 << 26), (1024, 1 << 20)):
        p = pool(page_size=ps)
        assert attention(lib, p, S=1, width=width) == 2
        assert append(lib, p, width=width, S=1, n=1) == 2
        assert compact(lib, p, S=1, width=width) == 2
        assert update(lib, p, n_in=1, n_out=1, width=width, ws_bytes=1 << 40) == 2


def test_null_pool(lib):
    assert lib.kvsel_paged_attention(None, 1, 1, P, P, 1, P, P, None, P, 1 << 30, None) == 1
    assert lib.kvsel_paged_attention_bytes(None, 1, 1) == -1
    assert lib.kvsel_pages_update_bytes(None, 1) == -1


@pytest.mark.parametrize("kw,status", [
    (dict(H=3), 1), (dict(H=0), 1), (dict(S=-1), 1), (dict(q=None), 1), (dict(q=ODD), 1),
    (dict(table=None), 1), (dict(width=0), 1), (dict(lens=None), 1), (dict(out=None), 1),
    (dict(out=ODD), 1), (dict(width=1 << 27), 2), (dict(S=8193), 2),
    (dict(S=8192, width=(1 << 17) + 1), 2),
])
def test_attention_rules(lib, kw, status):
    assert attention(lib, pool(), **kw) == status


def test_append_rules(lib):
    p = pool()
    for kw, status in [(dict(n=-1), 1), (dict(H=0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                       (dict(k=None), 1), (dict(v=None), 1), (dict(seqs=None, n=4), 1),
                       (dict(cache_pos=None), 1), (dict(q_out=None), 1), (dict(q_out=ODD), 1),
                       (dict(w=ODD), 1), (dict(q=rows(4096 + 8)), 1), (dict(k=rows(token=12)), 1),
                       (dict(v=rows(layer=-8)), 1), (dict(q=rows(None)), 1), (dict(rope=16, pos=None), 1),
                       (dict(rope=-16), 1), (dict(rope=20), 2), (dict(rope=144), 2), (dict(H=65532), 2),
                       (dict(width=0), 1), (dict(S=-1), 1), (dict(n=1 << 30, S=1), 2)]:
        assert append(lib, p, **kw) == status, kw


@pytest.mark.parametrize("kw,status", [
    (dict(most=-1), 1), (dict(rows_=-1), 1), (dict(S=-2), 1), (dict(lens=None), 1), (dict(idx=None), 1),
    (dict(offs=None), 1), (dict(table=None), 1), (dict(most=32769), 2), (dict(rows_=1 << 31), 2),
])
def test_compact_rules(lib, kw, status):
    assert compact(lib, pool(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_in=-1), 1), (dict(n_out=-1), 1), (dict(lens=None), 1), (dict(new=None), 1), (dict(ref=None), 1),
    (dict(parents=None, n_in=2), 1), (dict(ws=None), 1), (dict(ws=ODD), 1), (dict(ws_bytes=16), 1),
    (dict(out=None), 1), (dict(out=P), 1), (dict(out=ctypes.c_void_p(4096 + 56)), 1), (dict(width=1 << 27), 2),
])
def test_update_rules(lib, kw, status):
    assert update(lib, pool(), **kw) == status


def test_nothing_to_do(lib):
    p = pool()
    assert attention(lib, p, S=0, table=None, width=0, q=None, lens=None, out=None, ws=None,
                     ws_bytes=0) == 0
    assert append(lib, p, n=0, pos=None, cache_pos=None) == 0
    assert append(lib, p, q=None, k=None, v=None, H=0) == 0
    assert compact(lib, p, S=0) == 0
    assert compact(lib, p, rows_=0, idx=None) == 0
    assert compact(lib, p, most=0) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    ensure_built()
    from kv_cache_eviction_snapkv_gb300 import api
    K = torch.zeros((2, 4, 16, 2, 64))
    t = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        api.kvsel_paged_attention(torch.zeros((2, 1, 2, 64)), K, K, t, n)
    with pytest.raises(ValueError):
        api.kvsel_pages_update(K, K, t, n, n)
    with pytest.raises(ValueError):
        api.kvsel_paged_compact(K, K, t, n, torch.zeros((2, 1, 2), dtype=torch.int32), n, 1)
    with pytest.raises(ValueError):
        api.kvsel_paged_append(None, torch.zeros((2, 1, 2, 64)), torch.zeros((2, 1, 2, 64)), K, K, n)
