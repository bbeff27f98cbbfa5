"""The sampler on some of its rows: the others' logits are not looked at, their state and outputs stay."""
import numpy as np
import pytest
import torch

from nvfp4_w4a4_decode_gemv_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1000, 151936, 262208])
@pytest.mark.parametrize("top_p", [1.0, 0.9])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bool])
def test_only_the_named_rows_move(V, top_p, dtype):
    M, steps = 4, 11                                            # past the window of 8 entropies
    rng = np.random.default_rng(V)
    a, b = api.ResetSampler(M, V, top_p=top_p), api.ResetSampler(1, V, top_p=top_p)
    rows = torch.tensor([1, 0, 1, 0], device="cuda").to(dtype)
    a.token.fill_(77)
    for i in range(steps):
        x = torch.from_numpy((rng.standard_normal((M, V)) * 3).astype(np.float32)).cuda()
        u = torch.from_numpy(rng.random(M).astype(np.float32)).cuda()
        x[1] = float("nan")
        tok, H, T = a(x, None, u, rows=rows)
        one = b(x[2:3].contiguous(), None, u[2:3])              # row 2 as a row of its own
        for g, w in zip((tok, H, T), one):
            assert torch.equal(g[2:3], w)
        assert tok[[1, 3]].tolist() == [77, 77] and not H[[1, 3]].any() and not T[[1, 3]].any()
    stride = a.state.numel() // M
    fresh = api.ResetSampler(M, V).state.view(M, stride)
    assert torch.equal(a.state.view(M, stride)[[1, 3]], fresh[[1, 3]])
    assert torch.equal(a.state.view(M, stride)[2], b.state)
    # a row starts again, the others go on
    before = a.state.view(M, stride).clone()
    a.restart(torch.tensor([0, 0, 1, 0], device="cuda").to(dtype))
    after = a.state.view(M, stride)
    assert torch.equal(after[[0, 1, 3]], before[[0, 1, 3]]) and torch.equal(after[2], fresh[2])
    assert api.device_status() == 0


def test_row_masks_are_checked():
    s = api.ResetSampler(2, 100)
    x, u = torch.zeros((2, 100), device="cuda"), torch.zeros(2, device="cuda")
    for bad in (torch.ones(3, dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda"),
                torch.ones(2, dtype=torch.uint8), torch.ones(4, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="rows"):
            s(x, None, u, rows=bad)
        with pytest.raises(ValueError, match="rows"):
            s.restart(bad)
