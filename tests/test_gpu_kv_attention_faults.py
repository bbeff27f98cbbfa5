"""NaN and infinite queries, wherever the work is cut: a row without a finite softmax is NaN, never "saw no key"."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_kv_attention import _queries
from tests.test_gpu_kv_attention_modes import Pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("batch,rows,group,n", [(1, 1, 8, 40), (1, 1, 8, 6000), (8, 1, 8, 3000), (2, 3, 8, 9000), (1, 12, 16, 300),
                                                (2, 100, 8, 500), (1, 64, 8, 16000), (40, 40, 8, 700)])
@pytest.mark.parametrize("what", [np.nan, np.inf])
def test_rows_with_a_nan_or_infinite_query(D, batch, rows, group, n, what):
    """One element of a query of NaN gives NaN for that row and head, of infinity NaN too (every key's product with it
    is infinite or 0 times infinity); the other rows keep their bits."""
    rng = np.random.default_rng(n + rows)
    page, kvh = 64, 2
    p = Pool(rng, 100, page, kvh, D)
    table = torch.from_numpy(rng.integers(0, 100, (batch, -(-n // page))).astype(np.int32)).cuda()
    tokens, heads = batch * rows, group * kvh
    q = _queries(rng, tokens, heads, D, torch.bfloat16, 1.0)[0].cuda()
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * rows
    lse = torch.empty((tokens, heads), device="cuda")
    lse2 = torch.empty_like(lse)
    good = api.nvfp4_kv_attention(q, p.c, table, lens, cu, rows, lse=lse)
    assert torch.isfinite(good).all() and torch.isfinite(lse).all()
    hit = torch.zeros((tokens, heads), dtype=torch.bool, device="cuda")
    for t, h in ((0, 1), (tokens - 1, heads - 1), (tokens // 2, 0)):
        q[t, h, 5] = what
        hit[t, h] = True
    out = api.nvfp4_kv_attention(q, p.c, table, lens, cu, rows, lse=lse2)
    assert torch.isnan(out[hit]).all() and torch.isnan(lse2[hit]).all()
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse2[~hit], lse[~hit])
    assert api.device_status() == 0


@pytest.mark.parametrize("rows", [1, 4, 70])
def test_rows_that_see_nothing_stay_zero(rows):
    """... with or without a NaN query among them."""
    rng = np.random.default_rng(rows)
    p = Pool(rng, 10, 64, 1, 128)
    table = torch.zeros((2, 200), dtype=torch.int32, device="cuda")
    q = _queries(rng, 2 * rows, 8, 128, torch.bfloat16, 1.0)[0].cuda()
    q[0, 0, 0] = np.nan
    lens = torch.tensor([0, 6000], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    lse = torch.empty((2 * rows, 8), device="cuda")
    out = api.nvfp4_kv_attention(q, p.c, table, lens, cu, rows, lse=lse)
    assert not out[:rows].any() and np.isneginf(to_np(lse[:rows])).all() and torch.isfinite(out[rows:]).all()
