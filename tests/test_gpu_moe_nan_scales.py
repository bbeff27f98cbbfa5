"""A NaN among the scales of one token, one row of h or one row of weights: its own results are NaN, the bits of all others
stay."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import to_np
from tests.test_gpu_moe_experts import Case, _ids, _tensor

pytestmark = pytest.mark.gpu

NAN = 0x7F                                                        # of E4M3


def _same(got, want, other):
    """Bits equal where `other` is False, NaN where it is True."""
    nan = torch.isnan(got)
    assert torch.equal(nan, torch.from_numpy(other).cuda().expand(got.shape))
    assert torch.equal(torch.where(nan, 0.0, got.float()), torch.where(nan, 0.0, want.float()))


# SUM and copies of rows; rows laid out, one accumulator and (one expert takes most) two
@pytest.mark.parametrize("T,k,E", [(5, 2, 4), (64, 4, 9), (100, 2, 4), (300, 1, 2)])
def test_one_token(T, k, E):
    ids = _ids(np.random.default_rng(T), T, k, E)
    if k == 1:
        ids[::8] = 1 - ids[::8]
    c = Case(ids, E, 320, 192, seed=T)
    offsets, pairs, places = c.plan
    t = T // 2
    h, y = api.nvfp4_moe_gate_up(_tensor(c.x), c.up, c.routing), api.nvfp4_moe_down(_tensor(c.h), c.down, c.routing)
    x = _tensor(c.x)
    x.scales[t, 7] = NAN
    _same(api.nvfp4_moe_gate_up(x, c.up, c.routing), h, (pairs // k == t)[:, None])
    hq = _tensor(c.h)
    hq.scales[int(places[t, 0]), 3] = NAN
    _same(api.nvfp4_moe_down(hq, c.down, c.routing), y, (np.arange(T) == t)[:, None])
    assert api.device_status() == 0


@pytest.mark.parametrize("T,k,E", [(5, 2, 4), (100, 2, 4)])
def test_one_row_of_weights(T, k, E):
    c = Case(_ids(np.random.default_rng(T), T, k, E), E, 320, 192, seed=T)
    offsets, pairs, places = c.plan
    h, y = api.nvfp4_moe_gate_up(_tensor(c.x), c.up, c.routing), api.nvfp4_moe_down(_tensor(c.h), c.down, c.routing)
    e = int(c.ids[0, 0])
    of_e = np.zeros(T * k, bool)
    of_e[offsets[e]:offsets[e + 1]] = True
    for row in (70, 192 + 70):                                    # the gate's, the up's
        codes, scales = c.up_rows[0], c.up_rows[1].clone()
        scales[e, row, 5] = NAN
        w = api.nvfp4_moe_pack_weights(codes, scales, c.up.global_scale, True)
        _same(api.nvfp4_moe_gate_up(_tensor(c.x), w, c.routing), h, of_e[:, None] & (np.arange(192) == 70))
    codes, scales = c.down_rows[0], c.down_rows[1].clone()
    scales[e, 200, 11] = NAN
    w = api.nvfp4_moe_pack_weights(codes, scales, c.down.global_scale, False)
    _same(api.nvfp4_moe_down(_tensor(c.h), w, c.routing), y, (c.ids == e).any(1)[:, None] & (np.arange(320) == 200))
    assert api.device_status() == 0
