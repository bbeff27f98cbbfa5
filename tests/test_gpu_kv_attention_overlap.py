"""Row ranges that overlap because cu_q falls again: more work than a call of these sizes can have.  Nothing is computed,
the error is recorded, and the next call is as usual."""
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,tokens,n", [(129, 65536, 64000), (31, 65536, 128000), (300, 65536, 128000), (5, 12, 100),
                                            (200, 40, 64)])
def test_overlapping_row_ranges(batch, tokens, n):
    D, kvh, page = 64, 8, 1024
    c = api.NVFP4KVCache.empty(1, page, kvh, D)
    c.pages.zero_()
    table = torch.zeros((batch, -(-n // page)), dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    cu = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = tokens
    q = torch.zeros((tokens, kvh, D), dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 7.0)
    assert api.device_status() == 0
    api.nvfp4_kv_attention(q, c, table, lens, cu, max_q=1, out=out)
    assert api.device_status() == api.DEVERR_KV_RANGE
    assert torch.all(out == 7)
    # one request with a bad range, the others' ranges apart: those are served
    cu.fill_(0)
    cu[2:] = 3
    cu[1] = -1
    api.nvfp4_kv_attention(q, c, table, lens, cu, max_q=1, out=out)
    assert api.device_status() == api.DEVERR_KV_RANGE
    cu[1] = 0
    api.nvfp4_kv_attention(q, c, table, lens, cu, max_q=1, out=out)
    assert api.device_status() == 0 and not out[:3].any() and torch.all(out[3:] == 7)
