"""nvfp4_kv_plan refuses outputs that lie on its inputs or on one another (no GPU)."""
import os

import pytest

FAKE = 1 << 20
STEP = 1 << 16       # far apart: nothing overlaps unless it is the same


@pytest.fixture(scope="module")
def lib():
    from nvfp4_w4a4_decode_gemv_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def _call(lib, most=16, **p):
    names = ("ctx", "new", "table", "pages", "cnt", "out", "kv", "cu", "slots", "pos", "info")
    g = {n: p.get(n, FAKE + STEP * i) for i, n in enumerate(names)}
    return lib.nvfp4_kv_plan(g["ctx"], g["new"], 4, 64, g["table"], 8, g["pages"], 9, g["cnt"], g["out"], g["kv"], g["cu"],
                             g["slots"], g["pos"], most, g["info"], None)


def test_overlapping_outputs(lib):
    at = {n: FAKE + STEP * i for i, n in enumerate(("ctx", "new", "table", "pages", "cnt", "out", "kv", "cu", "slots", "pos",
                                                    "info"))}
    size = {"ctx": 16, "new": 16, "table": 128, "pages": 36, "cnt": 4, "out": 4, "kv": 16, "cu": 20, "slots": 64, "pos": 64,
            "info": 8}
    for a in ("table", "out", "kv", "cu", "slots", "pos", "info"):
        for b in at:
            if a == b or (a, b) in (("out", "cnt"), ("kv", "ctx")):
                continue
            assert _call(lib, **{a: at[b]}) == 2, (a, b)                       # the same start
            assert _call(lib, **{a: at[b] + size[b] - 4}) == 2, (a, b)         # the last entry
            assert _call(lib, **{a: at[b] - size[a] + 4}) == 2, (a, b)
    assert _call(lib, kv=at["ctx"] + 4) == 2 and _call(lib, kv=at["ctx"] - 4) == 2   # in place, or not at all
