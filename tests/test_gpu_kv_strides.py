"""Strides that no address uses: of a single token, of a single head."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.test_gpu_kv_attention import _cache, _queries
from tests.test_gpu_kv_cache import _rows

pytestmark = pytest.mark.gpu


def _odd(x, dim):
    """The same values with a stride of an odd number of elements along a dimension of size 1."""
    assert x.shape[dim] == 1
    strides = list(x.stride())
    strides[dim] = 1337
    return torch.as_strided(x, x.shape, strides)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,heads", [(1, 3), (5, 1), (1, 1)])
def test_append_and_attention(dtype, tokens, heads):
    rng = np.random.default_rng(tokens + heads)
    D, page = 128, 16
    dims = [d for d, n in enumerate((tokens, heads)) if n == 1]
    a, b = (_cache(np.random.default_rng(1), 4, page, heads, D)[0] for _ in range(2))
    k, v = _rows(rng, tokens, heads, D, dtype).cuda(), _rows(rng, tokens, heads, D, dtype).cuda()
    slots = torch.arange(tokens, dtype=torch.int32, device="cuda") + 20
    api.nvfp4_kv_append(k, v, slots, a)
    for d in dims:
        api.nvfp4_kv_append(_odd(k, d), _odd(v, d), slots, b)
    assert torch.equal(a.pages, b.pages)
    q = _queries(rng, tokens, heads, D, dtype, 1.0)[0].cuda()
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    args = (a, table, torch.tensor([50], dtype=torch.int32, device="cuda"), torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    want = api.nvfp4_kv_attention(q, *args)
    for d in dims:
        assert torch.equal(want, api.nvfp4_kv_attention(_odd(q, d), *args))
    assert api.device_status() == 0
