"""Refusals of the serving operators, at the C ABI and in the binding (no GPU): every bad argument comes back
before anything is launched."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20       # a 256-byte aligned non-NULL address; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from nvfp4_w4a4_decode_gemv_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def _cache(pages=FAKE, kg=FAKE, vg=FAKE, n=10, page=64, heads=8, dim=128):
    from nvfp4_w4a4_decode_gemv_gb300._lib import KVCacheDesc
    return KVCacheDesc(pages, kg, vg, n, page, heads, dim)


def test_page_bytes(lib):
    f = lib.nvfp4_kv_page_bytes
    assert f(64, 8, 128) == 64 * 8 * 144
    assert f(16, 1, 64) == 16 * 72
    for bad in ((0, 8, 128), (24, 8, 128), (1040, 8, 128), (64, 0, 128), (64, 1025, 128), (64, 8, 96), (64, 8, 256)):
        assert f(*bad) == 0


def test_release_refusals(lib):
    def call(lens=FAKE, ended=FAKE, batch=4, page=64, table=FAKE, width=8, pages=FAKE, cap=9, cnt=FAKE, out=FAKE):
        return lib.nvfp4_kv_release(lens, ended, batch, page, table, width, pages, cap, cnt, out, None)
    for null in ("lens", "ended", "table", "pages", "cnt", "out"):
        assert call(**{null: None}) == 1, null
    for bad in ({"batch": -1}, {"page": 20}, {"page": 0}, {"page": 2048}, {"width": -1}, {"cap": -1},
                {"batch": 1 << 20, "width": 1 << 20}):
        assert call(**bad) == 2, bad
    for bad in ("lens", "table", "pages", "cnt", "out"):
        assert call(**{bad: FAKE + 2}) == 3, bad


def test_plan_refusals(lib):
    names = ("ctx", "new", "table", "pages", "cnt", "out", "kv", "cu", "slots", "pos", "info")

    def call(batch=4, page=64, width=8, cap=9, most=16, **p):
        g = {n: p.get(n, FAKE) for n in names}
        return lib.nvfp4_kv_plan(g["ctx"], g["new"], batch, page, g["table"], width, g["pages"], cap, g["cnt"], g["out"],
                                 g["kv"], g["cu"], g["slots"], g["pos"], most, g["info"], None)
    for n in names:
        assert call(**{n: None}) == 1, n
        assert call(**{n: FAKE + 2}) == 3, n
    for bad in ({"batch": 0}, {"page": 8}, {"page": 72}, {"width": 0}, {"cap": -1}, {"most": -1},
                {"batch": 1 << 20, "width": 1 << 20}):
        assert call(**bad) == 2, bad


def _bad_caches():
    return [(_cache(pages=None), 1), (_cache(kg=None), 1), (_cache(vg=None), 1), (_cache(n=0), 2), (_cache(page=40), 2),
            (_cache(heads=0), 2), (_cache(dim=80), 2), (_cache(n=1 << 26, page=64), 2), (_cache(pages=FAKE + 8), 3),
            (_cache(kg=FAKE + 2), 3)]


def test_append_and_read_refusals(lib):
    c = _cache()

    def app(k=FAKE, v=FAKE, dtype=1, n=4, st=(1024, 128, 1024, 128), slots=FAKE, cache=c):
        return lib.nvfp4_kv_append(k, v, dtype, n, *st, slots, ctypes.byref(cache) if cache else None, None)

    def read(slots=FAKE, n=4, k=FAKE, v=FAKE, cache=c):
        return lib.nvfp4_kv_read(ctypes.byref(cache) if cache else None, slots, n, k, v, None)
    for bad, code in _bad_caches():
        assert app(cache=bad) == code and read(cache=bad) == code
    assert app(cache=None) == 1 and read(cache=None) == 1
    for null in ("k", "v", "slots"):
        assert app(**{null: None}) == 1 and read(**{null: None}) == 1
    assert app(dtype=2) == 4 and app(dtype=-1) == 4
    assert app(n=-1) == 2 and read(n=-1) == 2
    assert app(n=0) == 0 and read(n=0) == 0
    assert app(k=FAKE + 8) == 3 and app(v=FAKE + 4) == 3 and app(slots=FAKE + 1) == 3
    assert read(k=FAKE + 8) == 3 and read(v=FAKE + 8) == 3 and read(slots=FAKE + 2) == 3
    for i in range(4):
        st = [1024, 128, 1024, 128]
        st[i] += 4
        assert app(st=tuple(st)) == 3                       # BF16: 8 elements are 16 bytes
        assert app(st=tuple(st[:i] + [st[i] - 2] + st[i + 1:]), dtype=0) == 3


def test_attention_refusals(lib):
    c = _cache()
    need = lib.nvfp4_kv_attention_workspace_bytes(4, 4, 64, 8, 128)
    assert need > 0
    for bad in ((-1, 4, 64, 8, 128), (4, -1, 64, 8, 128), (4, 4, 60, 8, 128), (4, 4, 4, 8, 128), (4, 4, 8 * 65, 8, 128),
                (4, 4, 64, 8, 100)):
        assert lib.nvfp4_kv_attention_workspace_bytes(*bad) == 0, bad

    def call(q=FAKE, dtype=1, tokens=4, ts=8192, hs=128, heads=64, cache=c, table=FAKE, width=8, lens=FAKE, cu=None,
             batch=4, max_q=1, scale=0.1, window=0, out=FAKE, lse=None, ws=FAKE, wsb=need):
        return lib.nvfp4_kv_attention(q, dtype, tokens, ts, hs, heads, ctypes.byref(cache) if cache else None, table,
                                      width, lens, cu, batch, max_q, scale, window, out, lse, ws, wsb, None)
    for bad, code in _bad_caches():
        assert call(cache=bad) == code
    assert call(cache=None) == 1
    for null in ("q", "table", "lens", "out", "ws"):
        assert call(**{null: None}) == 1, null
    for bad in ({"dtype": 3}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")}, {"scale": float("inf")},
                {"window": -1}, {"max_q": 0}):
        assert call(**bad) == 4, bad
    for bad in ({"tokens": -1}, {"batch": -1}, {"width": 0}, {"tokens": 5}, {"heads": 12}, {"heads": 4},
                {"heads": 8 * 65}, {"wsb": need - 1}, {"width": 1 << 30}):
        assert call(**bad) == 2, bad
    for bad in ({"q": FAKE + 8}, {"out": FAKE + 8}, {"ws": FAKE + 16}, {"ts": 8196}, {"hs": 132}, {"lens": FAKE + 2},
                {"table": FAKE + 2}, {"cu": FAKE + 1}, {"lse": FAKE + 2}):
        assert call(**bad) == 3, bad
    assert call(tokens=0, batch=0) == 0 and call(tokens=0, cu=FAKE) == 0


def test_process_logits_refusals(lib):
    def call(x=FAKE, dtype=0, rows=4, V=1000, ld=1000, tok=FAKE, hist=10, nt=FAKE, npr=FAKE, rep=FAKE, pres=FAKE,
             freq=FAKE, ids=FAKE, vals=FAKE, nb=3, mask=FAKE, mc=4, mrows=FAKE, out=FAKE * 2):
        return lib.nvfp4_process_logits(x, dtype, rows, V, ld, tok, hist, nt, npr, rep, pres, freq, ids, vals, nb, mask,
                                        mc, mrows, float("-inf"), out, None)
    for null in ("x", "tok", "nt", "ids", "vals", "out"):
        assert call(**{null: None}) == 1, null
    for bad in ({"rows": -1}, {"rows": 65536}, {"V": 0}, {"V": (1 << 24) + 1, "ld": 1 << 25}, {"ld": 999}, {"hist": -1},
                {"nb": -1}, {"mc": 0}, {"mc": 3, "mrows": None}, {"out": FAKE, "dtype": 1}, {"out": FAKE, "ld": 1004}):
        assert call(**bad) == 2, bad
    assert call(dtype=2) == 4
    for bad in ("x", "tok", "nt", "npr", "rep", "pres", "freq", "ids", "vals", "mask", "mrows", "out"):
        assert call(**{bad: FAKE + 2 if bad != "x" else FAKE + 3}) == 3, bad
    assert call(rows=0) == 0


def test_binding_refuses_host_and_wrong_tensors():
    from nvfp4_w4a4_decode_gemv_gb300 import api
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    f32 = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError):
        api.NVFP4KVCache(torch.zeros((2, 1, 1, 18 * 128), dtype=torch.uint8), f32(1), f32(1))     # not on the GPU
    with pytest.raises(ValueError):
        api.NVFP4KVCache.empty(2, 24, 1, 128, device="cpu")
    with pytest.raises(ValueError):
        api.nvfp4_kv_plan(i32(2), i32(2), i32(2, 4), i32(9), i32(1), 16, 8)
    with pytest.raises(ValueError):
        api.nvfp4_kv_release(i32(2), torch.zeros(2, dtype=torch.uint8), i32(2, 4), i32(9), i32(1), 16)
    with pytest.raises(ValueError):
        api.nvfp4_process_logits(f32(2, 8))
