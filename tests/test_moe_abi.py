"""Refusals of the expert operators and of the rotating append, at the C ABI and in the binding (no GPU): every bad
argument comes back before anything is launched."""
import ctypes

import pytest
import torch

from tests.test_serving_abi import FAKE, _bad_caches, _cache, lib  # noqa: F401


def _router(top_k=8, score=0, groups=1, top_groups=1, group_best=1, renormalize=1, scale=1.0):
    from nvfp4_w4a4_decode_gemv_gb300._lib import MoERouter
    return MoERouter(top_k, score, groups, top_groups, group_best, renormalize, scale)


def test_route_refusals(lib):  # noqa: F811
    need = lib.nvfp4_moe_route_workspace_bytes(1000, 64)
    assert need > 0 and lib.nvfp4_moe_route_workspace_bytes(8, 64) == 0

    def call(x=FAKE, dtype=0, T=1000, E=64, ld=64, r=None, bias=None, rows=None, ids=FAKE, w=FAKE, off=FAKE, pairs=FAKE,
             places=FAKE, ws=FAKE, wsb=need, **router):
        r = _router(**router) if r is None else r
        return lib.nvfp4_moe_route(x, dtype, T, E, ld, ctypes.byref(r) if r else None, bias, rows, ids, w, off, pairs,
                                   places, ws, wsb, None)
    assert call(r=False) == 1
    for null in ("x", "ids", "w", "off", "pairs", "places", "ws"):
        assert call(**{null: None}) == 1, null
    for bad in ({"E": 0, "ld": 0}, {"E": 513, "ld": 513}, {"T": -1}, {"T": 1 << 30}, {"ld": 63}, {"top_k": 0}, {"top_k": 33},
                {"top_k": 65}, {"groups": 0}, {"groups": 3}, {"groups": 64}, {"groups": 8, "top_groups": 9},
                {"groups": 8, "top_groups": 0}, {"groups": 32, "top_groups": 3}, {"wsb": need - 1}):
        assert call(**bad) == 2, bad
    for bad in ({"dtype": 2}, {"score": 2}, {"score": -1}, {"group_best": 0}, {"group_best": 3}, {"scale": float("nan")},
                {"scale": float("inf")}):
        assert call(**bad) == 4, bad
    for bad in ("bias", "ids", "w", "off", "pairs", "places", "ws"):
        assert call(**{bad: FAKE + 2}) == 3, bad
    assert call(x=FAKE + 2) == 3 and call(x=FAKE + 1, dtype=1) == 3


def test_plan_refusals(lib):  # noqa: F811
    def call(ids=FAKE, T=4, k=2, E=8, off=FAKE, pairs=FAKE, places=FAKE, ws=None, wsb=0):
        return lib.nvfp4_moe_plan(ids, T, k, E, off, pairs, places, ws, wsb, None)
    for null in ("ids", "off", "pairs", "places"):
        assert call(**{null: None}) == 1, null
    for bad in ({"E": 0}, {"E": 513}, {"T": -1}, {"k": 0}, {"k": 33}, {"T": 1 << 30}):
        assert call(**bad) == 2, bad
    assert call(T=1000) == 1 and call(T=1000, ws=FAKE) == 2
    for bad in ("ids", "off", "pairs", "places"):
        assert call(**{bad: FAKE + 1}) == 3, bad


def test_pack_refusals(lib):  # noqa: F811
    f = lib.nvfp4_moe_packed_weight_bytes
    assert f(4, 128, 256, 0) == 4 * 18432 and f(1, 129, 320, 0) == 4 * 18432 and f(2, 256, 64, 1) == 4 * 18432
    for bad in ((0, 128, 256, 0), (513, 128, 256, 0), (1, 0, 256, 0), (1, (1 << 20) + 1, 256, 0), (1, 128, 32, 0),
                (1, 128, 96, 0), (1, 64, 256, 1), (1, 192, 256, 1), (1, 128, (1 << 20) + 64, 0)):
        assert f(*bad) == 0, bad

    def call(wq=FAKE, ws=FAKE, E=4, N=128, K=256, gated=0, p=FAKE, pb=4 * 18432):
        return lib.nvfp4_moe_pack_weights(wq, ws, E, N, K, gated, p, pb, None)
    for null in ("wq", "ws", "p"):
        assert call(**{null: None}) == 1, null
    assert call(pb=4 * 18432 - 1) == 2 and call(K=100) == 2 and call(N=64, gated=1) == 2
    assert call(wq=FAKE + 8) == 3 and call(ws=FAKE + 2) == 3 and call(p=FAKE + 8) == 3


def test_products_refusals(lib):  # noqa: F811
    def up(xq=FAKE, xs=FAKE, xg=FAKE, T=4, k=2, off=FAKE, pairs=FAKE, w=FAKE, wg=FAKE, E=8, I=64, K=256, h=FAKE,
           ws=None, wsb=0):
        return lib.nvfp4_moe_gate_up(xq, xs, xg, T, k, off, pairs, w, wg, E, I, K, h, ws, wsb, None)

    def down(xq=FAKE, xs=FAKE, xg=FAKE, T=4, k=2, off=FAKE, pairs=FAKE, places=FAKE, wt=FAKE, w=FAKE, wg=FAKE, E=8, N=100,
             K=256, y=FAKE, ws=None, wsb=0):
        return lib.nvfp4_moe_down(xq, xs, xg, T, k, off, pairs, places, wt, w, wg, E, N, K, y, ws, wsb, None)
    common = ("xq", "xs", "xg", "off", "pairs", "w", "wg")
    for null in common:
        assert up(**{null: None}) == 1 and down(**{null: None}) == 1, null
    assert up(h=None) == 1 and down(y=None) == 1 and down(places=None) == 1 and down(wt=None) == 1
    for bad in ({"T": -1}, {"k": 0}, {"k": 33}, {"T": 1 << 30}, {"E": 0}, {"E": 513}, {"K": 96}, {"K": 0}):
        assert up(**bad) == 2 and down(**bad) == 2, bad
    assert up(I=32) == 2 and up(I=96) == 2 and up(I=(1 << 19) + 64) == 2 and down(N=0) == 2 and down(N=(1 << 20) + 1) == 2
    assert up(T=0) == 0 and down(T=0) == 0
    for bad, by in (("xq", 8), ("xs", 2), ("xg", 2), ("off", 2), ("pairs", 1), ("w", 8), ("wg", 2)):
        assert up(**{bad: FAKE + by}) == 3 and down(**{bad: FAKE + by}) == 3, bad
    assert up(h=FAKE + 8) == 3 and down(y=FAKE + 8) == 3 and down(places=FAKE + 2) == 3 and down(wt=FAKE + 2) == 3
    for f, need in ((down, lib.nvfp4_moe_down_workspace_bytes(1000, 2, 8, 100, 256)),
                    (up, lib.nvfp4_moe_gate_up_workspace_bytes(1000, 2, 8, 256))):
        assert need > 0
        assert f(T=1000) == 1 and f(T=1000, ws=FAKE, wsb=need - 1) == 2 and f(T=1000, ws=FAKE + 8, wsb=need) == 3
    assert lib.nvfp4_moe_down_workspace_bytes(64, 2, 8, 100, 256) == 0
    assert lib.nvfp4_moe_gate_up_workspace_bytes(64, 2, 8, 256) == 0
    for bad in ((1000, 0, 8, 100, 256), (1000, 2, 0, 100, 256), (1000, 2, 8, 0, 256), (1000, 2, 8, 100, 32), (1 << 30, 2, 8, 100, 256)):
        assert lib.nvfp4_moe_down_workspace_bytes(*bad) == 0, bad


def test_rotating_append_refusals(lib):  # noqa: F811
    c = _cache()

    def call(q=FAKE, k=FAKE, v=FAKE, dtype=1, T=4, H=64, st=(8192, 128, 1024, 128, 1024, 128), pos=FAKE, table=FAKE, P=100,
             rot=128, style=0, slots=FAKE, cache=c, out=FAKE):
        return lib.nvfp4_kv_append_rope(q, k, v, dtype, T, H, *st, pos, table, P, rot, style, slots,
                                        ctypes.byref(cache) if cache else None, out, None)
    for bad, code in _bad_caches():
        assert call(cache=bad) == code
    assert call(cache=None) == 1
    for null in ("q", "k", "v", "pos", "table", "slots", "out"):
        assert call(**{null: None}) == 1, null
    for bad in ({"dtype": 2}, {"style": 2}, {"style": -1}):
        assert call(**bad) == 4, bad
    for bad in ({"T": -1}, {"H": -1}, {"H": 65537}, {"P": 0}, {"rot": 0}, {"rot": 16}, {"rot": 48}, {"rot": 160}):
        assert call(**bad) == 2, bad
    assert call(T=0) == 0
    assert call(H=0, q=None, out=None, table=FAKE + 8) == 3     # k and v alone: q is not looked at
    for bad, by in (("q", 8), ("k", 8), ("v", 8), ("table", 8), ("out", 8), ("slots", 2), ("pos", 2)):
        assert call(**{bad: FAKE + by}) == 3, bad
    for i in range(6):
        st = [8192, 128, 1024, 128, 1024, 128]
        st[i] += 4
        assert call(st=tuple(st)) == 3


def test_binding_refuses_host_and_wrong_tensors():
    from nvfp4_w4a4_decode_gemv_gb300 import api
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)
    for call in (lambda: api.nvfp4_moe_route(torch.zeros(2, 8), 2), lambda: api.nvfp4_moe_plan(i32(2, 2), 8),
                 lambda: api.MoERouting(i32(2, 2), None, i32(9), i32(4), i32(2, 2)),
                 lambda: api.nvfp4_moe_pack_weights(u8(1, 128, 128), u8(1, 128, 16), torch.zeros(1), False),
                 lambda: api.NVFP4MoEWeight(u8(18432), torch.zeros(1), 1, 128, 256, False),
                 lambda: api.nvfp4_moe_route(torch.zeros(2, 8), 2, score="tanh")):
        with pytest.raises(ValueError):
            call()
    t = api.rope_table(9, 32, device="cpu")
    assert t.shape == (9, 16, 2) and t.dtype == torch.float32 and t[0, :, 0].eq(1).all()
