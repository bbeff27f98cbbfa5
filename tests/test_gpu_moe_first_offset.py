"""A plan whose first expert's pairs do not begin at place 0: one without pairs, so that no row of h is left unwritten."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np
from tests.test_gpu_moe_experts import Case, _ids, _tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E", [(1, 4), (5, 4), (64, 4), (100, 4), (200, 512)])
def test_first_offset(T, E):
    c = Case(_ids(np.random.default_rng(T), T, 2, E), E, 128, 64)
    r = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), E, torch.from_numpy(c.weights).cuda())
    r.offsets[:] = r.offsets.clamp(min=1)                         # in order and within the pairs, but place 0 is no one's
    h, y = Guarded((2 * T, 64), torch.bfloat16), Guarded((T, 128), torch.float32)
    h.t.fill_(7.0)
    y.t.fill_(7.0)
    api.nvfp4_moe_gate_up(_tensor(c.x), c.up, r, out=h.t)
    assert api.device_status() == api.DEVERR_MOE_RANGE
    assert not to_np(h.t.float()).any()
    api.nvfp4_moe_down(_tensor(c.h), c.down, r, y=y.t)
    assert api.device_status() == api.DEVERR_MOE_RANGE
    assert not to_np(y.t).any()
    h.check("h")
    y.check("y")
    c.run()
