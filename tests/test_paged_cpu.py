"""Host-side refusals of the paged-cache entry points (no GPU needed): bad
arguments return their code before anything is launched."""
import ctypes

import pytest

from llama_decoder_forward_gb300 import build as B

P = 0x10000                       # a made-up device address; nothing reads it


@pytest.fixture(scope="module")
def S():
    B.build()
    from llama_decoder_forward_gb300 import smol
    return smol


def cache(S, **kw):
    f = dict(k_pages=P, v_pages=P, k_scale=None, v_scale=None, page_table=P, kv_dtype=S.KV_BF16, n_layers=2, n_pages=50,
             n_kv_heads=3, page_size=16, head_dim=64, max_pages=8)
    f.update(kw)
    return S._PagedCacheStruct(**f)


def chunk(S, **kw):
    f = dict(B=4, T=5, pos=P, row_start=None, n_new=None, rows=0)
    f.update(kw)
    return S._ChunkStruct(**f)


def rows(S, heads=3, hd=64, **kw):
    f = dict(data=P, layer=hd * heads * 20, seq=hd * heads * 5, row=hd * heads, head=hd)
    f.update(kw)
    return S._Rows(**f)


def append(S, c=None, k=None, r=None, r2=None, fn="smol_paged_append"):
    c, k, r, r2 = c or cache(S), k or chunk(S), r or rows(S), r2 or rows(S)
    return getattr(S.raw, fn)(*(ctypes.byref(x) for x in (c, k, r, r2)), None)


BAD_CACHE = [
    (dict(k_pages=None), -1), (dict(page_table=None), -1), (dict(kv_dtype=2), -1), (dict(kv_dtype=1), -1),
    (dict(n_layers=0), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1), (dict(max_pages=0), -1),
    (dict(head_dim=96), -2), (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=512), -2),
    (dict(max_pages=1 << 27), -2), (dict(v_pages=P + 8), -3), (dict(page_table=P + 2), -3),
    (dict(kv_dtype=1, k_scale=P, v_scale=P + 2), -3),
]
BAD_CHUNK = [
    (dict(pos=None), -1), (dict(B=0), -1), (dict(T=0), -1), (dict(row_start=P, n_new=P), -1),
    (dict(row_start=P, rows=-1), -1), (dict(pos=P + 1), -3), (dict(row_start=P, rows=1 << 31), -2),
    (dict(B=1 << 16, T=1 << 16), -2),
]


@pytest.mark.parametrize("fn", ["smol_paged_append", "smol_paged_read"])
def test_copies_refuse(S, fn):
    for kw, code in BAD_CACHE:
        assert append(S, c=cache(S, **kw), fn=fn) == code, kw
    for kw, code in BAD_CHUNK:
        assert append(S, k=chunk(S, **kw), fn=fn) == code, kw
    assert append(S, r=rows(S, data=None), fn=fn) == -1
    assert append(S, r=rows(S, data=P + 4), fn=fn) == -3
    assert append(S, r2=rows(S, row=100), fn=fn) == -3
    assert append(S, r2=rows(S, head=-64), fn=fn) == -1
    assert S.last_launch_count() == 0


def test_read_refuses_rows_on_one_another(S):
    for kw in (dict(head=32), dict(row=0), dict(layer=0), dict(seq=8)):
        assert append(S, r=rows(S, **kw), fn="smol_paged_read") == -1, kw
        assert append(S, r2=rows(S, **kw), fn="smol_paged_read") == -1, kw


def attend(S, c=None, layer=0, k=None, heads=9, q=None, o=None, scale=0.0, window=0, ws=P, n=1 << 40):
    c, k, q, o = c or cache(S), k or chunk(S), q or rows(S, heads=9), o or rows(S, heads=9)
    ref = ctypes.byref
    return S.raw.smol_paged_attention(ref(c), layer, ref(k), heads, ref(q), ref(o), scale, window, ws, n, None)


def test_attention_refuses(S):
    for kw, code in BAD_CACHE:
        assert attend(S, c=cache(S, **kw)) == code, kw
    for kw, code in BAD_CHUNK:
        assert attend(S, k=chunk(S, **kw)) == code, kw
    assert attend(S, layer=2) == -1 and attend(S, layer=-1) == -1
    assert attend(S, heads=10) == -2 and attend(S, heads=27) == -2 and attend(S, heads=0) == -1
    assert attend(S, k=chunk(S, B=4097, T=1)) == -2
    assert attend(S, window=-1) == -1
    for scale in (float("nan"), float("inf"), -1.0):
        assert attend(S, scale=scale) == -1
    assert attend(S, ws=None) == -1 and attend(S, ws=P + 8) == -3 and attend(S, n=16) == -5
    assert attend(S, o=rows(S, heads=9, head=32)) == -1 and attend(S, q=rows(S, heads=9, data=P + 2)) == -3
    assert S.last_launch_count() == 0


def test_workspace_query(S):
    size = lambda c, heads, b, t: S.raw.smol_paged_workspace_bytes(ctypes.byref(c), heads, b, t)
    assert size(cache(S), 9, 4, 5) >= 1024
    assert size(cache(S), 10, 4, 5) == 0 and size(cache(S), 9, 0, 5) == 0 and size(cache(S), 9, 4, 0) == 0
    assert size(cache(S, page_size=24), 9, 4, 5) == 0 and size(cache(S), 9, 5000, 1) == 0
