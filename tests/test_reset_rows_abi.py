"""Refusals of the sampler's calls for some rows, at the C ABI (no GPU)."""
import ctypes
import os

import pytest

FAKE = 1 << 20       # a 256-byte aligned non-NULL address; never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from nvfp4_w4a4_decode_gemv_gb300 import _lib, build
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return _lib.lib()


def test_refusals(lib):
    from nvfp4_w4a4_decode_gemv_gb300._lib import ResetParams
    p = ResetParams(0.6, 0.3, 1.0, 8)

    def call(logits=FAKE, M=4, V=1000, u=FAKE, rows=FAKE, state=FAKE, params=p, token=FAKE, ws=FAKE,
             wsb=lib.reset_workspace_bytes(4, 1000)):
        return lib.reset_sample_rows(logits, M, V, None, u, rows, state, ctypes.byref(params) if params else None, token,
                                     None, None, ws, wsb, None)
    for null in ("logits", "u", "rows", "state", "params", "token", "ws"):
        assert call(**{null: None}) == 1, null
    assert call(M=0) == 4 and call(M=65) == 4 and call(params=ResetParams(0.6, 0.3, 1.0, 0)) == 4
    assert call(V=0) == 2 and call(wsb=16) == 2
    for bad in ("logits", "u", "state", "token", "ws"):
        assert call(**{bad: FAKE + 2}) == 3, bad
    assert lib.reset_state_init_rows(None, 4, 8, FAKE, None) == 1
    assert lib.reset_state_init_rows(FAKE, 4, 8, None, None) == 1
    assert lib.reset_state_init_rows(FAKE, 0, 8, FAKE, None) == 4
    assert lib.reset_state_init_rows(FAKE, 4, 257, FAKE, None) == 4
    assert lib.reset_state_init_rows(FAKE + 8, 4, 8, FAKE, None) == 3
