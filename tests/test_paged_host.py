"""The paged cache's entry points without a GPU: the header, the exports and the structures
agree, bad arguments are refused before any CUDA call, and the binding checks its tensors."""
import ctypes
import os
import re

import pytest
import torch

from quantized_kv_attention_int4_b200 import abi, paged

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "flashloop_paged.h")
FAKE = 0x10000  # never dereferenced: every call below fails validation first


def index(**kw):
    f = dict(table=FAKE, length=FAKE, free_pages=FAKE, n_free=FAKE, status=None, slots=4, max_pages=8, pages=32)
    f.update(kw)
    return paged.fl_paged_index(*[f[n] for n, _ in paged.fl_paged_index._fields_])


def pool(**kw):
    f = dict(rec=FAKE, tail_k=FAKE, tail_v=FAKE, kv_heads=2, head_dim=128, page_tokens=64)
    f.update(kw)
    return paged.fl_paged_pool(*[f[n] for n, _ in paged.fl_paged_pool._fields_])


def ref(x):
    return ctypes.byref(x)


def test_header_and_binding_agree():
    text = open(HEADER).read()
    names = set(re.findall(r"^(?:fl_status|size_t)\s+(fl_\w+)\s*\(", text, re.M))
    assert names == set(paged.EXPORTED)
    for n in names:
        assert hasattr(paged.lib, n), n
    codes = {n: int(v) for n, v in re.findall(r"#define (FL_DEV_\w+) (\d+)", text)}
    assert len(codes) == 7
    for n, v in codes.items():
        assert getattr(paged, n) == v
    limits = {n: int(v) for n, v in re.findall(r"#define FL_PAGED_(\w+) (\d+)", text)}
    assert limits == {"MAX_BATCH": paged.MAX_BATCH, "MAX_SLOTS": paged.MAX_SLOTS, "MAX_BLOCKS": paged.MAX_BLOCKS,
                      "MAX_KEEP": paged.MAX_KEEP, "WS_HEAD": paged.WS_HEAD}
    assert ctypes.sizeof(paged.fl_paged_index) == 56 and ctypes.sizeof(paged.fl_paged_pool) == 40


@pytest.mark.parametrize("kw,st", [
    (dict(table=None), abi.FL_ERR_INVALID), (dict(length=None), abi.FL_ERR_INVALID),
    (dict(free_pages=None), abi.FL_ERR_INVALID), (dict(n_free=None), abi.FL_ERR_INVALID),
    (dict(table=FAKE + 2), abi.FL_ERR_INVALID), (dict(status=FAKE + 1), abi.FL_ERR_INVALID),
    (dict(slots=0), abi.FL_ERR_INVALID), (dict(max_pages=0), abi.FL_ERR_INVALID), (dict(pages=-1), abi.FL_ERR_INVALID),
    (dict(slots=paged.MAX_SLOTS + 1), abi.FL_ERR_UNSUPPORTED),
    (dict(max_pages=paged.MAX_BLOCKS + 1), abi.FL_ERR_UNSUPPORTED),
    (dict(pages=(1 << 25) - 1), abi.FL_ERR_UNSUPPORTED),  # places are 32-bit
])
def test_bad_indexes_are_refused_by_every_call(kw, st):
    x = index(**kw)
    assert paged._c_index_init(ref(x), None) == st
    assert paged._c_extend(ref(x), 1, None, FAKE, FAKE, FAKE, None) == st
    assert paged._c_release(ref(x), 1, None, None) == st
    assert paged._c_slot_map(ref(x), 1, None, FAKE, FAKE, 1, FAKE, FAKE, None) == st
    assert paged._c_append(ref(x), ref(pool()), 1, None, FAKE, FAKE, 1, FAKE, FAKE, 256, 128, None) == st
    assert paged._c_read(ref(x), ref(pool()), 1, FAKE, FAKE, FAKE, 256, 128, None) == st
    assert paged._c_ws_bytes(ref(x), ref(pool()), 1, 2) == 0
    assert paged._c_index_init(None, None) == abi.FL_ERR_INVALID


@pytest.mark.parametrize("kw,st", [
    (dict(rec=None), abi.FL_ERR_INVALID), (dict(tail_k=None), abi.FL_ERR_INVALID), (dict(tail_v=None), abi.FL_ERR_INVALID),
    (dict(rec=FAKE + 8), abi.FL_ERR_INVALID), (dict(tail_v=FAKE + 8), abi.FL_ERR_INVALID),
    (dict(kv_heads=0), abi.FL_ERR_INVALID), (dict(head_dim=64), abi.FL_ERR_UNSUPPORTED),
    (dict(page_tokens=32), abi.FL_ERR_UNSUPPORTED),
    (dict(kv_heads=1 << 20), abi.FL_ERR_UNSUPPORTED),  # rows are addressed with 32-bit coordinates
])
def test_bad_pools_are_refused(kw, st):
    x, p = index(), pool(**kw)
    assert paged._c_append(ref(x), ref(p), 1, None, FAKE, FAKE, 1, FAKE, FAKE, 256, 128, None) == st
    assert paged._c_read(ref(x), ref(p), 1, FAKE, FAKE, FAKE, 256, 128, None) == st
    assert paged._c_ws_bytes(ref(x), ref(p), 1, 2) == 0
    big = 1 << 40
    assert paged._c_select(ref(x), ref(p), 1, None, 2, FAKE, 256, 128, 3, FAKE, FAKE, big, None) == st
    assert paged._c_attn(ref(x), ref(p), 1, None, 2, FAKE, 256, 128, None, 0, FAKE, 256, 128, None, FAKE, big, None) == st


def test_index_calls_check_their_arguments():
    x = index()
    ext = lambda b=1, s=None, n=FAKE, st=FAKE, cu=FAKE: paged._c_extend(ref(x), b, s, n, st, cu, None)  # noqa: E731
    assert ext(b=-1) == abi.FL_ERR_INVALID
    assert ext(b=5) == abi.FL_ERR_INVALID                       # identity slots beyond the table
    assert ext(b=paged.MAX_BATCH + 1, s=FAKE) == abi.FL_ERR_UNSUPPORTED
    assert ext(n=None) == abi.FL_ERR_INVALID
    assert ext(st=None) == abi.FL_ERR_INVALID
    assert ext(cu=None) == abi.FL_ERR_INVALID
    assert ext(s=FAKE + 2) == abi.FL_ERR_INVALID
    assert paged._c_release(ref(x), -1, None, None) == abi.FL_ERR_INVALID
    assert paged._c_release(ref(x), 5, None, None) == abi.FL_ERR_INVALID
    assert paged._c_release(ref(x), 0, None, None) == abi.FL_OK
    smap = lambda b=1, t=4, st=FAKE, cu=FAKE, pl=FAKE, po=FAKE: paged._c_slot_map(ref(x), b, None, st, cu, t, pl, po, None)  # noqa: E731
    assert smap(t=-1) == abi.FL_ERR_INVALID
    assert smap(b=5) == abi.FL_ERR_INVALID
    assert smap(st=None) == abi.FL_ERR_INVALID
    assert smap(cu=None) == abi.FL_ERR_INVALID
    assert smap(pl=FAKE + 1) == abi.FL_ERR_INVALID
    assert smap(t=0) == abi.FL_OK and smap(b=0) == abi.FL_OK and smap(pl=None, po=None) == abi.FL_OK


def test_append_and_read_check_their_arguments():
    x, p = index(), pool()
    app = lambda b=1, t=4, st=FAKE, cu=FAKE, k=FAKE, v=FAKE, ts=256, hs=128: paged._c_append(  # noqa: E731
        ref(x), ref(p), b, None, st, cu, t, k, v, ts, hs, None)
    assert app(t=-1) == abi.FL_ERR_INVALID
    assert app(b=5) == abi.FL_ERR_INVALID
    assert app(st=None) == app(cu=None) == app(k=None) == app(v=None) == abi.FL_ERR_INVALID
    assert app(k=FAKE + 8) == abi.FL_ERR_INVALID                # not 16-byte aligned
    assert app(ts=250) == app(hs=100) == app(ts=-256) == abi.FL_ERR_INVALID
    assert app(t=0) == app(b=0) == abi.FL_OK                    # nothing to do, nothing enqueued
    rd = lambda t=4, pl=FAKE, k=FAKE, v=FAKE, ts=256, hs=128: paged._c_read(  # noqa: E731
        ref(x), ref(p), t, pl, k, v, ts, hs, None)
    assert rd(t=-1) == rd(pl=None) == rd(k=None) == rd(v=FAKE + 2) == abi.FL_ERR_INVALID
    assert rd(ts=64) == rd(hs=64) == rd(ts=128) == rd(ts=248) == abi.FL_ERR_INVALID   # output rows would overlap
    assert rd(ts=128, hs=504) == abi.FL_ERR_INVALID             # head by head: four rows of 128 reach into the next head
    assert rd(t=0) == abi.FL_OK


def test_append_refuses_more_work_than_it_counts():
    # two items per entry and per 64 tokens, for each head, in 32 bits
    x, p = index(), pool(kv_heads=32)
    app = lambda t: paged._c_append(ref(x), ref(p), 1, None, FAKE, FAKE, t, FAKE, FAKE + 8, 4096, 128, None)  # noqa: E731
    most = (2 ** 31 - 1 - 65536) // 64 - 1
    assert app(most * 64 + 63) == abi.FL_ERR_INVALID            # v is not aligned: the count itself passed
    assert app((most + 1) * 64) == abi.FL_ERR_UNSUPPORTED
    assert app(2 ** 31 - 1) == abi.FL_ERR_UNSUPPORTED


def test_attention_and_selection_check_their_arguments():
    x, p = index(), pool()
    ws = paged._c_ws_bytes(ref(x), ref(p), 3, 4)
    assert ws > paged.WS_HEAD
    att = lambda b=3, s=None, hq=4, q=FAKE, qb=512, qh=128, sel=None, keep=0, o=FAKE, ob=512, oh=128, lse=None, w=FAKE, n=ws: \
        paged._c_attn(ref(x), ref(p), b, s, hq, q, qb, qh, sel, keep, o, ob, oh, lse, w, n, None)  # noqa: E731
    assert att(b=-1) == att(b=5) == abi.FL_ERR_INVALID
    assert att(hq=3) == att(hq=0) == abi.FL_ERR_INVALID          # not a multiple of the key-value heads
    assert att(q=None) == att(q=FAKE + 8) == att(qb=500) == att(qh=-128) == abi.FL_ERR_INVALID
    assert att(o=None) == att(o=FAKE + 4) == att(ob=510) == att(oh=64) == att(ob=64) == abi.FL_ERR_INVALID
    assert att(ob=128) == att(ob=128, oh=376) == att(ob=508) == abi.FL_ERR_INVALID   # rows of two entries would overlap
    assert att(lse=FAKE + 2) == abi.FL_ERR_INVALID
    assert att(sel=FAKE, keep=0) == att(sel=FAKE + 1, keep=2) == abi.FL_ERR_INVALID
    assert att(sel=FAKE, keep=paged.MAX_KEEP + 1) == abi.FL_ERR_UNSUPPORTED
    assert att(w=None) == att(n=ws - 1) == att(w=FAKE + 16) == abi.FL_ERR_WORKSPACE
    assert att(b=0) == abi.FL_OK
    sel = lambda b=3, hq=4, q=FAKE, keep=2, out=FAKE, w=FAKE, n=ws: paged._c_select(  # noqa: E731
        ref(x), ref(p), b, None, hq, q, 512, 128, keep, out, w, n, None)
    assert sel(hq=5) == sel(q=None) == sel(keep=0) == sel(out=None) == sel(out=FAKE + 2) == abi.FL_ERR_INVALID
    assert sel(keep=paged.MAX_KEEP + 1) == abi.FL_ERR_UNSUPPORTED
    assert sel(n=ws - 1) == abi.FL_ERR_WORKSPACE
    assert sel(b=0) == abi.FL_OK
    # work units are counted in 32 bits
    wide = index(slots=8192, max_pages=paged.MAX_BLOCKS, pages=1 << 16)
    assert paged._c_ws_bytes(ref(wide), ref(pool(kv_heads=16)), 8192, 16) == 0
    assert paged._c_ws_init(None, 1 << 20, None) == paged._c_ws_init(FAKE, 100, None) == abi.FL_ERR_WORKSPACE


def test_binding_refuses_host_tensors_and_wrong_types():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedIndex(i(2, 3), i(2), i(6), i(1))
    with pytest.raises(ValueError, match="slots"):
        paged.PagedIndex(i(2), i(2), i(6), i(1))
    with pytest.raises(TypeError, match="int32"):
        paged.PagedIndex(i(2, 3).long(), i(2), i(6), i(1))
    rec = torch.zeros(4, 2, 9216, dtype=torch.uint8)
    tail = torch.zeros(2, 2, 64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="9216"):
        paged.PagedPool(rec[..., :9000], tail, tail)
    with pytest.raises(ValueError, match="tail_v"):
        paged.PagedPool(rec, tail, tail[:, :1])
    with pytest.raises(ValueError, match="same shape"):
        paged.PagedPool(rec, tail, tail[:1])
    with pytest.raises(ValueError, match="CUDA"):
        paged.PagedPool(rec, tail, tail)
