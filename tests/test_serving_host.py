"""Refusals of the serving operators on a paged cache, before anything is launched (no GPU
needed: the pointers are never dereferenced)."""
import pytest

import exact_io_aware_70_b200 as ea

P = 0x10000
INV, UNS, ALI = ea.ATTN_ERR_INVALID_ARG, ea.ATTN_ERR_UNSUPPORTED, ea.ATTN_ERR_ALIGNMENT


def _call(fn, ok, kw):
    a = dict(ok, **kw)
    assert set(a) == set(ok)
    return fn(*a.values(), None)


TABLES = dict(ctx=P, new=P, free=P, head=P, head_out=P, table=P, seq=P, cu=P, slots=P, B=4, T=10,
              num_free=5, page_size=16, max_pages=8, num_pages=50)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, INV) for k in list(TABLES)[:9]], *[({k: P + 2}, ALI) for k in list(TABLES)[:9]],
    (dict(slots=P + 4), ALI), (dict(B=0), INV), (dict(B=8193), UNS), (dict(T=0), INV),
    (dict(T=2 ** 30 + 1), INV), (dict(num_free=0), INV), (dict(page_size=8), INV),
    (dict(page_size=48), INV), (dict(page_size=2048), INV), (dict(max_pages=0), INV),
    (dict(max_pages=2 ** 27), INV), (dict(num_pages=0), INV),
])
def test_tables_refusals(kw, code):
    assert _call(ea.lib.attn_page_tables, TABLES, kw) == code


APPEND = dict(k=P, v=P, slots=P, kc=P, vc=P, kb=P, T=4, Hkv=2, d=128, stride=256, page_size=16,
              num_pages=50)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, INV) for k in ("k", "v", "slots", "kc", "vc")],
    *[({k: P + 8}, ALI) for k in ("k", "v", "kc", "vc", "kb")], (dict(slots=P + 4), ALI),
    (dict(T=0), INV), (dict(Hkv=0), INV), (dict(Hkv=65536), INV), (dict(d=96), UNS),
    (dict(stride=255), INV), (dict(stride=0), INV), (dict(stride=260), ALI),
    (dict(page_size=100), INV), (dict(num_pages=0), INV), (dict(num_pages=2 ** 30), INV),
])
def test_append_refusals(kw, code):
    assert _call(ea.lib.attn_paged_append, APPEND, kw) == code


FWD = dict(q=P, kc=P, vc=P, table=P, cu=P, seq=P, o=P, lse=P, B=2, T=4, Hq=8, Hkv=2, d=128,
           stride=1024, page_size=16, max_pages=8, num_pages=50, causal=1, scale=0.1, ws=P,
           ws_bytes=ea.attn_fwd_paged_workspace_bytes(128))


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, INV) for k in ("q", "kc", "vc", "table", "cu", "seq", "o", "lse", "ws")],
    *[({k: P + 8}, ALI) for k in ("q", "kc", "vc", "o")],
    *[({k: P + 2}, ALI) for k in ("table", "cu", "seq", "lse")], (dict(ws=P + 128), ALI),
    (dict(B=0), INV), (dict(T=0), INV), (dict(Hq=7), INV), (dict(Hq=0), INV), (dict(Hkv=0), INV),
    (dict(Hq=258), UNS), (dict(d=80), UNS), (dict(stride=1016), INV), (dict(stride=1028), ALI),
    (dict(stride=2 ** 40), INV), (dict(page_size=24), INV), (dict(max_pages=0), INV),
    (dict(num_pages=0), INV), (dict(causal=2), INV), (dict(scale=0.0), INV),
    (dict(scale=float("inf")), INV), (dict(scale=float("nan")), INV),
    (dict(ws_bytes=FWD["ws_bytes"] - 1), INV),
])
def test_fwd_paged_refusals(kw, code):
    if "stride" not in kw and kw.get("Hq", 0) > 8:
        kw = dict(kw, stride=kw["Hq"] * 128)
    assert _call(ea.lib.attn_fwd_paged, FWD, kw) == code


SPARSE = dict(q=P, kc=P, vc=P, table=P, cu=P, seq=P, sel=P, o=P, lse=P, B=2, T=4, Hq=8, Hkv=2,
              d=64, K=4, stride=512, page_size=16, max_pages=8, num_pages=50, scale=0.1, ws=P,
              ws_bytes=ea.attn_fwd_paged_workspace_bytes(64))


@pytest.mark.parametrize("kw,code", [
    (dict(sel=None), INV), (dict(q=None), INV), (dict(sel=P + 2), ALI), (dict(K=0), INV),
    (dict(K=481), UNS), (dict(K=61, page_size=1024), UNS), (dict(ws_bytes=0), INV),
    (dict(o=P + 2), ALI), (dict(Hq=9), INV), (dict(scale=-1.0), INV),
])
def test_sparse_refusals(kw, code):
    assert _call(ea.lib.attn_sparse_paged, SPARSE, kw) == code


SELECT = dict(q=P, kb=P, table=P, cu=P, seq=P, sel=P, B=2, T=4, Hq=8, Hkv=2, d=64, K=4, first=1,
              last=1, stride=512, page_size=16, max_pages=8, num_pages=50, ws=P,
              ws_bytes=ea.attn_page_select_workspace_bytes(4, 2, 8))


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, INV) for k in ("q", "kb", "table", "cu", "seq", "sel", "ws")],
    *[({k: P + 8}, ALI) for k in ("q", "kb", "ws")],
    *[({k: P + 2}, ALI) for k in ("table", "cu", "seq", "sel")],
    (dict(K=0), INV), (dict(first=-1), INV), (dict(last=-1), INV), (dict(first=3, last=2), INV),
    (dict(max_pages=16385), UNS), (dict(ws_bytes=SELECT["ws_bytes"] - 1), INV), (dict(d=32), UNS),
    (dict(Hq=2 * 129, stride=129 * 128), UNS), (dict(stride=504), INV), (dict(T=0), INV),
])
def test_select_refusals(kw, code):
    assert _call(ea.lib.attn_page_select, SELECT, kw) == code


def test_workspace_sizes():
    assert ea.attn_fwd_paged_workspace_bytes(96) == 0
    assert ea.attn_fwd_paged_workspace_bytes(64) % 256 == 0
    assert 0 < ea.attn_fwd_paged_workspace_bytes(64) < ea.attn_fwd_paged_workspace_bytes(128)
    assert ea.attn_page_select_workspace_bytes(0, 2, 8) == 0
    assert ea.attn_page_select_workspace_bytes(4, 2, 8) > 0


def test_python_wrappers_refuse_wrong_tensors():
    import torch
    x = torch.zeros((4, 8, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    cache = torch.zeros((5, 2, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):      # not on a GPU
        ea.attn_paged_append(x[:, :2], x[:, :2], i.long(), cache, cache)
    with pytest.raises((TypeError, ValueError)):
        ea.attn_fwd_paged([1], cache, cache, i[None], i, i, x, x, True, 0.1, i)
