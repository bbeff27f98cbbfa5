"""The binding's workspaces: a caller's own is looked at, the binding's own is ready on the stream of the call."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_kv_attention import _cache, _queries, _table

pytestmark = pytest.mark.gpu


def _call(rng, batch=2, n=3000, kvh=2, heads=16, D=128, page=64):
    c, _, _, _ = _cache(rng, 64, page, kvh, D)
    t = torch.from_numpy(rng.integers(0, 64, (batch, -(-n // page))).astype(np.int32)).cuda()
    q = _queries(rng, batch, heads, D, torch.bfloat16, 1.0)[0].cuda()
    return q, c, t, torch.full((batch,), n, dtype=torch.int32, device="cuda")


def test_a_callers_workspace_is_checked():
    args = _call(np.random.default_rng(1))
    need = api.nvfp4_kv_attention_workspace_bytes(2, 2, 16, 2, 128)
    want = api.nvfp4_kv_attention(*args)
    zeros = lambda n, **kw: torch.zeros(n, **{"dtype": torch.uint8, "device": "cuda", **kw})
    for bad in (zeros(need, device="cpu"), zeros(2 * need)[::2], zeros(need, dtype=torch.float32)):
        with pytest.raises(ValueError, match="workspace"):
            api.nvfp4_kv_attention(*args, workspace=bad)
    with pytest.raises(RuntimeError, match="SHAPE"):
        api.nvfp4_kv_attention(*args, workspace=zeros(need - 1))
    assert torch.equal(want, api.nvfp4_kv_attention(*args, workspace=zeros(need)))
