"""Plans that do not hold together, for every number of tokens: what has no product is zero, whatever the workspace held."""
import numpy as np
import pytest
import torch

from oracle import moe as O
from nvfp4_w4a4_decode_gemv_gb300 import api
from tests.gpu_util import Guarded, to_np
from tests.test_gpu_moe_experts import Case, _ids, _tensor

pytestmark = pytest.mark.gpu


def _down(c, r):
    """y over a workspace full of NaN."""
    need = max(16, api.nvfp4_moe_down_workspace_bytes(c.T, c.k, c.E, c.hidden, c.inter))
    ws, y = Guarded((need,), torch.uint8), Guarded((c.T, c.hidden), torch.float32)
    ws.t.fill_(0xFF)
    api.nvfp4_moe_down(_tensor(c.h), c.down, r, y=y.t, workspace=ws.t)
    y.check("y")
    ws.check("workspace")
    return y.t


@pytest.mark.parametrize("T,E", [(4, 4), (64, 300), (65, 4), (100, 4), (130, 512), (400, 16)])
@pytest.mark.parametrize("broken", ["alternating", "negative", "beyond"])
def test_refused_offsets_give_zero(T, E, broken):
    c = Case(_ids(np.random.default_rng(T), T, 2, E), E, 128, 64)
    r = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), E, torch.from_numpy(c.weights).cuda())
    if broken == "alternating":
        r.offsets[::2], r.offsets[1::2] = 0, 2 * T
    else:
        r.offsets[E // 2 if broken == "negative" else E] = -3 if broken == "negative" else 2 * T + 1
    y = _down(c, r)
    assert api.device_status() == api.DEVERR_MOE_RANGE
    assert not to_np(y).any()
    c.check_down(_down(c, c.routing))                             # the plan as it was
    assert api.device_status() == 0


@pytest.mark.parametrize("T", [65, 100, 500])
def test_places_behind_the_last_pair_are_skipped(T):
    """Beyond 64 tokens y goes by the places: those that no pair stands at have no product."""
    rng = np.random.default_rng(T)
    ids = _ids(rng, T, 3, 6)
    ids[ids == 2] = -1
    c = Case(ids, 6, 192, 64, seed=1)
    offsets, pairs, places = c.plan
    last, P = int(offsets[-1]), 3 * T
    assert 0 < last < P
    r = api.nvfp4_moe_plan(torch.from_numpy(c.ids).cuda(), 6, torch.from_numpy(c.weights).cuda())
    places = places.copy()
    for (t, j), at in {(0, 0): last, (1, 2): P - 1, (T - 1, 1): P, (7, 0): -2}.items():
        r.places[t, j], places[t, j] = at, -1
    c.plan = offsets, pairs, places
    c.check_down(_down(c, r))
    assert api.device_status() == api.DEVERR_MOE_RANGE
