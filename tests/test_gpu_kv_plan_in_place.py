"""The plan's new lengths over the old ones, and the refusal of outputs that lie on other arguments."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_kv_plan import _case, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [1, 8, 257, 1000, 2500])
@pytest.mark.parametrize("most_new", [1, 90, 700])
@pytest.mark.parametrize("count_in_place", [False, True])
def test_lengths_in_place(batch, most_new, count_in_place):
    """kv_lens is ctx_lens: one CTA or many, the same result as with two arrays."""
    rng = np.random.default_rng(batch + most_new)
    page = 32
    ctx, new, table, stack, count = _case(rng, batch, page, 300, most_new, 0 if batch % 2 else -(batch // 3))
    most = int(new.sum())
    want = S.kv_plan(ctx, new, table, stack, count, page, most)
    for _ in range(3):
        t, cnt, lens = _dev(table), _dev([count]), _dev(ctx)
        out = api.KVPlan.empty(batch, most, "cuda", cnt if count_in_place else None)
        out.kv_lens = lens
        api.nvfp4_kv_plan(lens, _dev(new), t, _dev(stack), cnt, page, out=out)
        got = (t, out.slots, out.positions, out.cu_q, lens, out.free_count, out.info)
        for g, w, name in zip(got, want, ("table", "slots", "positions", "cu_q", "kv_lens", "free_count", "info")):
            assert np.array_equal(to_np(g).reshape(-1), np.asarray(w).reshape(-1)), name
